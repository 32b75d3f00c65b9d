// api_window_sink.cu -- C entry points of the sliding-window attention with sinks: argument checks,
// tensor maps and dispatch (the kernels are the window instances of the prefill and backward, and
// decode_sink_sm100.cu).

#include "diffattn_v2.h"
#include "internal.h"

namespace {

using bf16 = __nv_bfloat16;

int status_of(cudaError_t e) { return e == cudaSuccess ? DA2_OK : DA2_ERR_CUDA; }

bool map(CUtensorMap* m, const void* base, int H, int S, int B, uint32_t rows) {
  return da2::encode_bshd_bf16(m, base, 128, static_cast<uint64_t>(H), static_cast<uint64_t>(S),
                               static_cast<uint64_t>(B), 64, rows) == cudaSuccess;
}

// Prefill of [B,S] tensors, or with cu_seqlens of `total` packed tokens (S: the longest sequence).
// o_branch and lse: both (training) or neither.
int prefill(const void* q, const void* k, const void* v, const float* lambda, void* out, float* o_branch, float* lse,
            bool train, const int32_t* cu_seqlens, int B, int S, int total, int Hq, int Hkv, int D, int window,
            int sink, da2_stream_t stream) {
  const bool packed = total >= 0;
  if (B < 0 || S < 0 || D <= 0 || !da2::paired_heads(Hq, Hkv) || window < 1 || sink < 0) return DA2_ERR_INVALID;
  if (B == 0 || S == 0 || total == 0) return DA2_OK;
  for (const void* p : {q, k, v, static_cast<const void*>(lambda), static_cast<const void*>(out)})
    if (!p || !da2::is_aligned(p, 16)) return DA2_ERR_INVALID;
  if (train && (!o_branch || !lse || !da2::is_aligned(o_branch, 16) || !da2::is_aligned(lse, 16))) return DA2_ERR_INVALID;
  if (packed && (!cu_seqlens || !da2::is_aligned(cu_seqlens, 4))) return DA2_ERR_INVALID;
  if (D != 128) return DA2_ERR_UNSUPPORTED;
  const long long tiles = (static_cast<long long>(S) + 127) / 128;
  if (tiles > 65535 || tiles * B * (Hq / 2) > 2147483647LL) return DA2_ERR_UNSUPPORTED;
  int* err = nullptr;
  if (da2::device_error_word(&err) != cudaSuccess) return DA2_ERR_CUDA;
  const int rows = packed ? total : S, batch = packed ? 1 : B;
  CUtensorMap tq, tk, tv, to;
  if (!map(&tq, q, Hq, rows, batch, 128) || !map(&tk, k, Hkv, rows, batch, 128) || !map(&tv, v, Hkv, rows, batch, 128) ||
      da2::encode_out_bf16(&to, out, D, Hq / 2, rows, batch) != cudaSuccess)
    return DA2_ERR_CUDA;
  // a window of S or more keys, or as many sinks, is the plain causal mask
  const bool causal = window >= S || sink >= S;
  return status_of(da2::launch_prefill(tq, tk, tv, nullptr, to, lambda, static_cast<bf16*>(out), err, B, S, Hq, Hkv, 1,
                                       causal ? 0 : window, packed ? cu_seqlens : nullptr,
                                       reinterpret_cast<cudaStream_t>(stream), nullptr, lse, sink,
                                       train ? o_branch : nullptr));
}

int backward(const void* q, const void* k, const void* v, const float* lambda, const float* o_branch,
             const float* lse, const void* dout, void* dq, void* dk, void* dv, float* dlambda,
             const int32_t* cu_seqlens, int B, int S, int total, int Hq, int Hkv, int D, int window, int sink,
             void* workspace, size_t workspace_bytes, da2_stream_t stream) {
  const bool packed = total >= 0;
  if (B < 0 || S < 0 || D <= 0 || !da2::paired_heads(Hq, Hkv) || window < 1 || sink < 0) return DA2_ERR_INVALID;
  if (B == 0 || S == 0 || total == 0) return DA2_OK;
  for (const void* p : {q, k, v, static_cast<const void*>(lambda), static_cast<const void*>(o_branch),
                        static_cast<const void*>(lse), dout, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv),
                        static_cast<const void*>(dlambda), static_cast<const void*>(workspace)})
    if (!p || !da2::is_aligned(p, 16)) return DA2_ERR_INVALID;
  if (packed && (!cu_seqlens || !da2::is_aligned(cu_seqlens, 4))) return DA2_ERR_INVALID;
  const size_t need = packed ? diffattn_v2_backward_varlen_window_sink_workspace_size(B, S, total, Hq, Hkv, window, sink)
                             : diffattn_v2_backward_window_sink_workspace_size(B, S, Hq, Hkv, window, sink);
  if (workspace_bytes < need) return DA2_ERR_INVALID;
  if (D != 128) return DA2_ERR_UNSUPPORTED;
  // grid limits: 128-row tiles on grid y; the preprocess runs 4 (row, pair) warps per CTA
  const long long padded = packed ? static_cast<long long>(total) + 128LL * B + 128
                                  : static_cast<long long>(B) * (static_cast<long long>(S) + 128);
  // (and the parts of the tiles that hold sinks beside them)
  if ((static_cast<long long>(S) + 127) / 128 > 60000 || padded > 2147483647LL ||
      padded * (Hq / 2) > 4LL * 2147483647LL || static_cast<long long>(B) * Hq > 2147483647LL)
    return DA2_ERR_UNSUPPORTED;
  // The tile kernel's CTAs are counted in an int, and every sequence has those of the longest one: at
  // most half of this product for dQ, as many for the key tiles, and for the parts of split tiles
  // about 600 per 64-row query block of the longest sequence (72e6 of those).
  if ((static_cast<long long>(S) + 127) / 128 * B * Hq > 2000000000LL) return DA2_ERR_UNSUPPORTED;
  int* err = nullptr;
  if (da2::device_error_word(&err) != cudaSuccess) return DA2_ERR_CUDA;
  const int rows = packed ? total : S, batch = packed ? 1 : B;
  CUtensorMap q64, q128, o64, o128, k64, k128, v64, v128;
  if (!map(&q64, q, Hq, rows, batch, 64) || !map(&q128, q, Hq, rows, batch, 128) ||
      !map(&o64, dout, Hq / 2, rows, batch, 64) || !map(&o128, dout, Hq / 2, rows, batch, 128) ||
      !map(&k64, k, Hkv, rows, batch, 64) || !map(&k128, k, Hkv, rows, batch, 128) ||
      !map(&v64, v, Hkv, rows, batch, 64) || !map(&v128, v, Hkv, rows, batch, 128))
    return DA2_ERR_CUDA;
  const bool causal = window >= S || sink >= S;
  return status_of(da2::launch_backward_sm100(
      q64, q128, o64, o128, k64, k128, v64, v128, lambda, nullptr, lse, static_cast<const bf16*>(dout),
      static_cast<bf16*>(dq), static_cast<bf16*>(dk), static_cast<bf16*>(dv), dlambda, static_cast<float*>(workspace),
      err, B, S, Hq, Hkv, 1, reinterpret_cast<cudaStream_t>(stream), packed ? cu_seqlens : nullptr,
      packed ? total : 0, causal ? 0 : window, sink, o_branch));
}

int decode(const void* q, const void* kcache, const void* vcache, const int32_t* block_table, const int32_t* seqlens,
           const float* lambda, void* out, int B, int Smax, int max_pages, int page_shift, int num_pages, int Hq,
           int Hkv, int D, int window, int sink, da2_stream_t stream) {
  for (const void* p : {q, kcache, vcache, static_cast<const void*>(lambda), static_cast<const void*>(out)})
    if (!p || !da2::is_aligned(p, 16)) return DA2_ERR_INVALID;
  if (!seqlens || !da2::is_aligned(seqlens, 4)) return DA2_ERR_INVALID;
  const int group = Hq / Hkv;
  if (D != 128 || !(group == 2 || group == 4 || group == 8 || group == 16)) return DA2_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > 65535) return DA2_ERR_UNSUPPORTED;
  int* err = nullptr;
  if (da2::device_error_word(&err) != cudaSuccess) return DA2_ERR_CUDA;
  const int rows = block_table ? 1 << page_shift : Smax, batch = block_table ? num_pages : B;
  CUtensorMap tk, tv;
  const uint32_t tokens = block_table && rows < 16 ? 8 : 16;
  if (da2::encode_kv_halves(&tk, kcache, Hkv, rows, batch, tokens) != cudaSuccess ||
      da2::encode_kv_halves(&tv, vcache, Hkv, rows, batch, tokens) != cudaSuccess)
    return DA2_ERR_CUDA;
  return status_of(da2::launch_decode_sink(tk, tv, static_cast<const bf16*>(q), seqlens, lambda,
                                           static_cast<bf16*>(out), err, B, Smax, Hq, Hkv,
                                           window < Smax ? window : Smax, sink < Smax ? sink : Smax, block_table,
                                           max_pages, page_shift, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int diffattn_v2_prefill_window_sink(const void* q, const void* k, const void* v, const float* lambda, void* out, int B,
                                    int S, int Hq, int Hkv, int D, int window, int sink, da2_stream_t stream) {
  return prefill(q, k, v, lambda, out, nullptr, nullptr, false, nullptr, B, S, -1, Hq, Hkv, D, window, sink, stream);
}

int diffattn_v2_prefill_varlen_window_sink(const void* q, const void* k, const void* v, const float* lambda, void* out,
                                           const int32_t* cu_seqlens, int B, int max_seqlen, int total_tokens, int Hq,
                                           int Hkv, int D, int window, int sink, da2_stream_t stream) {
  if (total_tokens < 0) return DA2_ERR_INVALID;
  return prefill(q, k, v, lambda, out, nullptr, nullptr, false, cu_seqlens, B, max_seqlen, total_tokens, Hq, Hkv, D,
                 window, sink, stream);
}

int diffattn_v2_prefill_window_sink_train(const void* q, const void* k, const void* v, const float* lambda, void* out,
                                          float* o_branch, float* lse, int B, int S, int Hq, int Hkv, int D, int window,
                                          int sink, da2_stream_t stream) {
  return prefill(q, k, v, lambda, out, o_branch, lse, true, nullptr, B, S, -1, Hq, Hkv, D, window, sink, stream);
}

int diffattn_v2_prefill_varlen_window_sink_train(const void* q, const void* k, const void* v, const float* lambda,
                                                 void* out, float* o_branch, float* lse, const int32_t* cu_seqlens,
                                                 int B, int max_seqlen, int total_tokens, int Hq, int Hkv, int D,
                                                 int window, int sink, da2_stream_t stream) {
  if (total_tokens < 0) return DA2_ERR_INVALID;
  return prefill(q, k, v, lambda, out, o_branch, lse, true, cu_seqlens, B, max_seqlen, total_tokens, Hq, Hkv, D, window,
                 sink, stream);
}

size_t diffattn_v2_backward_window_sink_workspace_size(int B, int S, int Hq, int Hkv, int window, int sink) {
  if (B <= 0 || S <= 0 || !da2::paired_heads(Hq, Hkv) || window < 1 || sink < 0) return 0;
  return da2::backward_sink_workspace_bytes(B, S, 0, Hq, Hkv, window, sink, false);
}

size_t diffattn_v2_backward_varlen_window_sink_workspace_size(int B, int max_seqlen, int total_tokens, int Hq, int Hkv,
                                                              int window, int sink) {
  if (B <= 0 || max_seqlen <= 0 || total_tokens <= 0 || !da2::paired_heads(Hq, Hkv) || window < 1 || sink < 0) return 0;
  return da2::backward_sink_workspace_bytes(B, max_seqlen, total_tokens, Hq, Hkv, window, sink, true);
}

int diffattn_v2_backward_window_sink(const void* q, const void* k, const void* v, const float* lambda,
                                     const float* o_branch, const float* lse, const void* dout, void* dq, void* dk,
                                     void* dv, float* dlambda, int B, int S, int Hq, int Hkv, int D, int window,
                                     int sink, void* workspace, size_t workspace_bytes, da2_stream_t stream) {
  return backward(q, k, v, lambda, o_branch, lse, dout, dq, dk, dv, dlambda, nullptr, B, S, -1, Hq, Hkv, D, window, sink,
                  workspace, workspace_bytes, stream);
}

int diffattn_v2_backward_varlen_window_sink(const void* q, const void* k, const void* v, const float* lambda,
                                            const float* o_branch, const float* lse, const void* dout, void* dq,
                                            void* dk, void* dv, float* dlambda, const int32_t* cu_seqlens, int B,
                                            int max_seqlen, int total_tokens, int Hq, int Hkv, int D, int window,
                                            int sink, void* workspace, size_t workspace_bytes, da2_stream_t stream) {
  if (total_tokens < 0) return DA2_ERR_INVALID;
  return backward(q, k, v, lambda, o_branch, lse, dout, dq, dk, dv, dlambda, cu_seqlens, B, max_seqlen, total_tokens, Hq,
                  Hkv, D, window, sink, workspace, workspace_bytes, stream);
}

int diffattn_v2_decode_window_sink(const void* q, const void* kcache, const void* vcache, const int32_t* seqlens,
                                   const float* lambda, void* out, int B, int Smax, int Hq, int Hkv, int D, int window,
                                   int sink, da2_stream_t stream) {
  if (B < 0 || Smax <= 0 || D <= 0 || !da2::paired_heads(Hq, Hkv) || window < 1 || sink < 0) return DA2_ERR_INVALID;
  if (Smax > (1 << 30)) return DA2_ERR_INVALID;
  if (B == 0) return DA2_OK;
  return decode(q, kcache, vcache, nullptr, seqlens, lambda, out, B, Smax, 0, 0, 0, Hq, Hkv, D, window, sink, stream);
}

int diffattn_v2_decode_paged_window_sink(const void* q, const void* kpages, const void* vpages,
                                         const int32_t* block_table, const int32_t* seqlens, const float* lambda,
                                         void* out, int B, int max_pages, int page_size, int num_pages, int Hq, int Hkv,
                                         int D, int window, int sink, da2_stream_t stream) {
  const int shift = da2::page_shift_of(page_size);
  if (B < 0 || max_pages <= 0 || num_pages <= 0 || D <= 0 || !da2::paired_heads(Hq, Hkv) || window < 1 || sink < 0 ||
      shift < 0)
    return DA2_ERR_INVALID;
  if (static_cast<long long>(max_pages) * page_size > (1LL << 30)) return DA2_ERR_INVALID;
  if (B == 0) return DA2_OK;
  if (!block_table || !da2::is_aligned(block_table, 4)) return DA2_ERR_INVALID;
  return decode(q, kpages, vpages, block_table, seqlens, lambda, out, B, max_pages * page_size, max_pages, shift,
                num_pages, Hq, Hkv, D, window, sink, stream);
}

}  // extern "C"
