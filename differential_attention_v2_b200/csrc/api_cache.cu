// api_cache.cu -- C entry points of the rotary positions and of the paged cache's pages: argument
// checks and dispatch to rope.cu and cache_pages.cu.

#include "diffattn_v2.h"
#include "internal.h"

namespace {

int status_of(cudaError_t e) { return e == cudaSuccess ? DA2_OK : DA2_ERR_CUDA; }

size_t size_of(int dtype) { return dtype == DA2_DTYPE_F32 ? 4 : 2; }

// The checks and parameters that both rotary entry points share.
int rope_common(da2::RopeParams* p, const int32_t* positions, const float* inv_freq, const int* sections, int n_axes,
                int T, int Hq, int Hkv, int D, int dtype, int interleaved, int inverse) {
  if (T < 0 || Hq <= 0 || Hkv < 0 || D <= 0 || D % 2 != 0 || n_axes < 1 || !sections) return DA2_ERR_INVALID;
  if ((dtype != DA2_DTYPE_BF16 && dtype != DA2_DTYPE_F32) || (interleaved & ~1) || (inverse & ~1)) return DA2_ERR_INVALID;
  if (n_axes > 4 || D > 4096 || Hq > 65536 || Hkv > 65536) return DA2_ERR_UNSUPPORTED;
  long long P = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0) return DA2_ERR_INVALID;
    P += sections[a];
    if (P > D / 2) return DA2_ERR_INVALID;
    p->sec_end[a] = static_cast<int>(P);
  }
  if (P < 1) return DA2_ERR_INVALID;
  if (T > 0 && (!positions || !inv_freq || !da2::is_aligned(positions, 4) || !da2::is_aligned(inv_freq, 4)))
    return DA2_ERR_INVALID;
  p->positions = positions;
  p->inv_freq = inv_freq;
  p->n_axes = n_axes;
  p->P = static_cast<int>(P);
  p->T = T;
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->D = D;
  p->interleaved = interleaved;
  p->inverse = inverse;
  return DA2_OK;
}

// (2^30 pages and tokens: page and token numbers plus a CTA's stride stay inside an int)
bool pool_ok(int B, int max_pages, int page_shift, int num_pages) {
  return B >= 0 && max_pages > 0 && page_shift >= 0 && num_pages > 0 && num_pages <= (1 << 30) &&
         (static_cast<long long>(max_pages) << page_shift) <= (1LL << 30);
}

template <typename... P>
bool ints_ok(const P*... p) {
  return ((p != nullptr && da2::is_aligned(p, 4)) && ...);
}

}  // namespace

extern "C" {

int diffattn_v2_rope(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions,
                     const float* inv_freq, const int* sections, int n_axes, int T, int Hq, int Hkv, int D,
                     int64_t q_stride, int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride, int dtype,
                     int interleaved, int inverse, da2_stream_t stream) {
  da2::RopeParams p = {};
  const int st = rope_common(&p, positions, inv_freq, sections, n_axes, T, Hq, Hkv, D, dtype, interleaved, inverse);
  if (st != DA2_OK || T == 0) return st;
  const size_t el = size_of(dtype);
  const int64_t wq = static_cast<int64_t>(Hq) * D, wk = static_cast<int64_t>(Hkv) * D;
  if (!q || !q_out || !da2::is_aligned(q, el) || !da2::is_aligned(q_out, el) || q_stride < wq || q_out_stride < wq)
    return DA2_ERR_INVALID;
  if (Hkv > 0 && (!k || !k_out || !da2::is_aligned(k, el) || !da2::is_aligned(k_out, el) || k_stride < wk || k_out_stride < wk))
    return DA2_ERR_INVALID;
  p.q = q;
  p.q_out = q_out;
  p.q_stride = q_stride;
  p.qo_stride = q_out_stride;
  if (Hkv > 0) {
    p.k = k;
    p.k_out = k_out;
    p.k_stride = k_stride;
    p.ko_stride = k_out_stride;
  }
  if (da2::bounds_error_word(&p.err) != cudaSuccess) return DA2_ERR_CUDA;
  return status_of(da2::launch_rope(p, dtype == DA2_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream)));
}

int diffattn_v2_rope_append_paged(const void* q, const void* k, const void* v, void* q_out, const int32_t* positions,
                                  const float* inv_freq, const int* sections, int n_axes, void* kpages, void* vpages,
                                  const int32_t* block_table, const int32_t* seqlens, const int32_t* cu_seqlens, int T,
                                  int B, int max_pages, int page_size, int num_pages, int Hq, int Hkv, int D,
                                  int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t q_out_stride, int dtype,
                                  int interleaved, da2_stream_t stream) {
  da2::RopeParams p = {};
  p.page_shift = da2::page_shift_of(page_size);
  if (Hkv <= 0 || !pool_ok(B, max_pages, p.page_shift, num_pages)) return DA2_ERR_INVALID;
  const int st = rope_common(&p, positions, inv_freq, sections, n_axes, T, Hq, Hkv, D, dtype, interleaved, 0);
  if (st != DA2_OK || T == 0) return st;
  const size_t el = size_of(dtype);
  const int64_t wq = static_cast<int64_t>(Hq) * D, wk = static_cast<int64_t>(Hkv) * D;
  for (const void* x : {q, k, v, static_cast<const void*>(q_out), static_cast<const void*>(kpages),
                        static_cast<const void*>(vpages)})
    if (!x || !da2::is_aligned(x, el)) return DA2_ERR_INVALID;
  if (q_stride < wq || q_out_stride < wq || k_stride < wk || v_stride < wk) return DA2_ERR_INVALID;
  if (!ints_ok(block_table, seqlens) || !da2::is_aligned(cu_seqlens, 4)) return DA2_ERR_INVALID;
  if (!cu_seqlens && T != B) return DA2_ERR_INVALID;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out = q_out;
  p.k_out = kpages;
  p.v_out = vpages;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.qo_stride = q_out_stride;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.cu_seqlens = cu_seqlens;
  p.B = B;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  if (da2::bounds_error_word(&p.err) != cudaSuccess) return DA2_ERR_CUDA;
  return status_of(da2::launch_rope(p, dtype == DA2_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream)));
}

int diffattn_v2_cache_extend(int32_t* block_table, int32_t* seqlens, int32_t* refs, const int32_t* n_new,
                             int32_t* result, int B, int max_pages, int page_size, int num_pages,
                             da2_stream_t stream) {
  const int shift = da2::page_shift_of(page_size);
  if (!pool_ok(B, max_pages, shift, num_pages)) return DA2_ERR_INVALID;
  if (B == 0) return DA2_OK;
  if (!ints_ok(block_table, seqlens, refs, n_new, result)) return DA2_ERR_INVALID;
  // (the pages that all sequences ask for are summed in an int)
  if (B > da2::kMaxCacheSeqs || static_cast<long long>(B) * max_pages > 2147483647LL) return DA2_ERR_UNSUPPORTED;
  return status_of(da2::launch_cache_extend(block_table, seqlens, refs, n_new, result, B, max_pages, shift, num_pages,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

int diffattn_v2_cache_fork(int32_t* block_table, int32_t* seqlens, int32_t* refs, const int32_t* parents,
                           const int32_t* children, int32_t* copies, int32_t* result, int n, int B, int max_pages,
                           int page_size, int num_pages, da2_stream_t stream) {
  const int shift = da2::page_shift_of(page_size);
  if (n < 0 || !pool_ok(B, max_pages, shift, num_pages)) return DA2_ERR_INVALID;
  if (n == 0) return DA2_OK;
  if (!ints_ok(refs, parents, children, result) || !copies || !da2::is_aligned(copies, 8)) return DA2_ERR_INVALID;
  if (B > 0 && !ints_ok(block_table, seqlens)) return DA2_ERR_INVALID;  // (a table without rows is not read)
  if (n > da2::kMaxCacheSeqs) return DA2_ERR_UNSUPPORTED;
  return status_of(da2::launch_cache_fork(block_table, seqlens, refs, parents, children, copies, result, n, B, max_pages,
                                          shift, num_pages, reinterpret_cast<cudaStream_t>(stream)));
}

int diffattn_v2_cache_trim(int32_t* block_table, const int32_t* seqlens, int32_t* refs, int32_t* result, int B,
                           int max_pages, int page_size, int num_pages, int window, int sink, da2_stream_t stream) {
  const int shift = da2::page_shift_of(page_size);
  if (!pool_ok(B, max_pages, shift, num_pages) || window < 1 || sink < 0) return DA2_ERR_INVALID;
  if (B == 0) return DA2_OK;
  if (!ints_ok(block_table, seqlens, refs, result)) return DA2_ERR_INVALID;
  return status_of(da2::launch_cache_trim(block_table, seqlens, refs, result, B, max_pages, shift, num_pages, window,
                                          sink, reinterpret_cast<cudaStream_t>(stream)));
}

int diffattn_v2_cache_free(int32_t* block_table, int32_t* seqlens, int32_t* refs, const int32_t* seqs, int32_t* result,
                           int n, int B, int max_pages, int num_pages, da2_stream_t stream) {
  if (n < 0 || !pool_ok(B, max_pages, 0, num_pages)) return DA2_ERR_INVALID;
  if (n == 0) return DA2_OK;
  if (!ints_ok(refs, seqs, result) || (B > 0 && !ints_ok(block_table, seqlens))) return DA2_ERR_INVALID;
  return status_of(da2::launch_cache_free(block_table, seqlens, refs, seqs, result, n, B, max_pages, num_pages,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int diffattn_v2_cache_compact(const int32_t* block_table, const int32_t* refs, int32_t* block_table_out,
                              int32_t* refs_out, int32_t* moves, int32_t* result, int B, int max_pages, int num_pages,
                              da2_stream_t stream) {
  if (!pool_ok(B, max_pages, 0, num_pages)) return DA2_ERR_INVALID;
  if (!ints_ok(refs, refs_out, result)) return DA2_ERR_INVALID;
  if (B > 0 && !ints_ok(block_table, block_table_out)) return DA2_ERR_INVALID;
  if (num_pages > 1 && (!moves || !da2::is_aligned(moves, 8))) return DA2_ERR_INVALID;
  return status_of(da2::launch_cache_compact(block_table, refs, block_table_out, refs_out, moves, result, B, max_pages,
                                             num_pages, reinterpret_cast<cudaStream_t>(stream)));
}

int diffattn_v2_cache_copy_pages(void* kpages, void* vpages, const int32_t* copies, int n, int num_pages,
                                 size_t page_bytes, da2_stream_t stream) {
  if (n < 0 || num_pages <= 0 || page_bytes == 0) return DA2_ERR_INVALID;
  if (n == 0) return DA2_OK;
  if (!kpages || !vpages || kpages == vpages || !copies || !da2::is_aligned(copies, 8)) return DA2_ERR_INVALID;
  if (!da2::is_aligned(kpages, 16) || !da2::is_aligned(vpages, 16)) return DA2_ERR_INVALID;
  if (page_bytes % 16 != 0 || page_bytes / 16 > 0x40000000u) return DA2_ERR_UNSUPPORTED;
  return status_of(da2::launch_cache_copy_pages(kpages, vpages, copies, n, num_pages, page_bytes,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
