// internal.h -- host-side launchers shared between the C ABI (api.cu) and the kernel files.
// Not installed; the public interface is include/diffattn_v2.h.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace da2 {

// Host-side argument checks shared by the entry points of api_window_sink.cu and api_cache.cu.
inline bool is_aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
// Hq even and the heads of every pair inside one KV group
inline bool paired_heads(int Hq, int Hkv) { return Hq > 0 && Hkv > 0 && Hq % 2 == 0 && Hq % (2LL * Hkv) == 0; }
// a page size that paged caches have: a power of two from 8 to 4096; its log2, or -1
inline int page_shift_of(int page_size) {
  if (page_size < 8 || page_size > 4096 || (page_size & (page_size - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

// Launches a kernel that begins with pdl_wait(), so that the launch overlaps the end of the kernel
// before it in the stream; cluster > 0 gives the cluster's size. Passes called one after the other, us,
// with and without: one user's decode 6.0 and 8.2, five page operations 22.8 and 32.8, rotary append of
// 64 tokens 5.1 and 6.2, packed training step 114 and 125. (Letting the next kernel in as soon as this
// one's CTAs run fills the SMs with waiting CTAs: rotary of 2,049 tokens 9.8 and 7.5 us with that before
// and after the wait, 5.0 without.)
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t stream,
                           const A&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  // (the call's own status: a failed launch takes its error with it, or the next launch would report it)
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

// bf16 prefill on tcgen05 (D = 128); window > 0 (causal only) limits query i to keys
// i-window+1 .. i. With cu_seqlens (device, B+1 entries) the tensors hold B packed sequences
// as one [1,T] batch and S is the longest sequence. Tensor maps: Q over [B,S,Hq,D], K/V over [B,S,Hkv,D],
// boxes of 64 (d) x 1 (head) x 128 (rows) x 1, 128-byte swizzle; tmKh (optional) over K with
// boxes of 64 (d) x 1 x 64 (rows) x 1, for the CTA-pair form (GQA groups of a multiple of 4);
// tmO over out [B,S,Hq/2,D] (with cu_seqlens [1,T,Hq/2,D]) from encode_out_bf16. sink > 0 (with a
// window): keys 0 .. sink-1 stay visible; the training forward then writes O_b in fp32.
cudaError_t launch_prefill(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                           const CUtensorMap* tmKh, const CUtensorMap& tmO, const float* lambda, __nv_bfloat16* out, int* err, int B, int S,
                           int Hq, int Hkv, int causal, int window, const int* cu_seqlens, cudaStream_t stream,
                           __nv_bfloat16* o_branch = nullptr, float* lse = nullptr, int sink = 0,
                           float* o_branch_f32 = nullptr);

// The [B,S] bf16 prefill with the V2 lambda computed in the kernel:
// lambda[t, p] = sigmoid(x[t] . w_t[p] + bias[p]) with x [B*S, d_model] and w_t [Hq/2, d_model]
// bf16 (d_model a multiple of 8), bias fp32 [Hq/2] or null; lambda_out (fp32 [B*S, Hq/2]) gets
// a copy when not null. Tensor maps as for launch_prefill.
cudaError_t launch_prefill_lambda_fused(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                        const CUtensorMap& tmO, const __nv_bfloat16* x, const __nv_bfloat16* w_t,
                                        const float* bias, float* lambda_out, int d_model, __nv_bfloat16* out,
                                        int* err, int B, int S, int Hq, int Hkv, int causal, cudaStream_t stream);

// tcgen05 backward of the bf16 prefill (D = 128): preprocess into the workspace (row terms;
// backward_stats_bytes, or backward_varlen_workspace_bytes with packed sequences), then the
// dK/dV and dQ tile kernels. Tensor maps over q [B,S,Hq,D], dout [B,S,Hq/2,D], k and v
// [B,S,Hkv,D] with 64- and 128-row boxes (64 d x 1 head). With cu_seqlens (device, B+1
// entries) the tensors hold B packed sequences as one [1,T] batch (T = total_tokens) and S
// is the longest sequence. window > 0 (causal only): query i saw keys i-window+1 .. i. With
// o_branch_f32 the sink form: keys 0 .. sink-1 too (o_branch unused).
size_t backward_stats_bytes(int B, int S, int Hq);
size_t backward_varlen_workspace_bytes(int B, int T, int Hq);
// the sink form's workspace (T: total tokens of packed sequences)
size_t backward_sink_workspace_bytes(int B, int S, int T, int Hq, int Hkv, int window, int sink, bool packed);
cudaError_t launch_backward_sm100(const CUtensorMap& tmQ64, const CUtensorMap& tmQ128, const CUtensorMap& tmO64,
                                  const CUtensorMap& tmO128, const CUtensorMap& tmK64, const CUtensorMap& tmK128,
                                  const CUtensorMap& tmV64, const CUtensorMap& tmV128, const float* lambda,
                                  const __nv_bfloat16* o_branch, const float* lse, const __nv_bfloat16* dout,
                                  __nv_bfloat16* dq, __nv_bfloat16* dk, __nv_bfloat16* dv, float* dlambda,
                                  float* workspace, int* err, int B, int S, int Hq, int Hkv, int causal,
                                  cudaStream_t stream, const int32_t* cu_seqlens = nullptr, int total_tokens = 0,
                                  int window = 0, int sink = 0, const float* o_branch_f32 = nullptr);

// bf16 decode (D = 128): split kernel + combine. Tensor maps over the caches [B,Smax,Hkv,D],
// boxes of 64 (d) x 1 x 64 (tokens) x 1, 128-byte swizzle. With block_table the maps cover
// pages [num_pages, 1 << page_shift, Hkv, D] with boxes of min(page_size, 64) tokens and
// Smax = max_pages << page_shift. T new tokens per sequence (q [B,T,Hq,D]); T * Hq/Hkv <= 16.
cudaError_t launch_decode(const CUtensorMap& tmK, const CUtensorMap& tmV, const __nv_bfloat16* q,
                          const int32_t* seqlens, const float* lambda, __nv_bfloat16* out, float* ws_o,
                          float* ws_ml, int* counters, int* err, int B, int Smax, int Hq, int Hkv, int nsplit,
                          int split_len, const int32_t* block_table, int max_pages, int page_shift, int T,
                          cudaStream_t stream, int window = 0);

// bf16 decode step (D = 128) over the last `window` and the first `sink` keys of each sequence:
// one cluster per (KV head, sequence), no workspace. tmK, tmV from encode_kv_halves over the cache
// (boxes of 16 tokens) or the pages (boxes of min(page_size, 16) tokens).
cudaError_t launch_decode_sink(const CUtensorMap& tmK, const CUtensorMap& tmV, const __nv_bfloat16* q,
                               const int32_t* seqlens, const float* lambda, __nv_bfloat16* out, int* err, int B,
                               int Smax, int Hq, int Hkv, int window, int sink, const int32_t* block_table,
                               int max_pages, int page_shift, cudaStream_t stream);

// 5-D bf16 tensor map over a row-major [B,S,H,128] cache as (64 of d, token, half of d, head, b), box
// {64, tokens, 2, 1, 1}, 128-byte swizzle: one copy brings both halves of a token run of one head.
cudaError_t encode_kv_halves(CUtensorMap* map, const void* base, uint64_t H, uint64_t S, uint64_t B, uint32_t tokens);

// Page bookkeeping of a paged cache (cache_pages.cu): one cluster each; block tables
// [B, max_pages], refs [num_pages]; result one int. At most kMaxCacheSeqs sequences (extend) or
// pairs (fork).
constexpr int kMaxCacheSeqs = 2048;
cudaError_t launch_cache_extend(int32_t* table, int32_t* seqlens, int32_t* refs, const int32_t* n_new,
                                int32_t* result, int B, int max_pages, int page_shift, int num_pages,
                                cudaStream_t stream);
cudaError_t launch_cache_fork(int32_t* table, int32_t* seqlens, int32_t* refs, const int32_t* parents,
                              const int32_t* children, int32_t* copies, int32_t* result, int n, int B, int max_pages,
                              int page_shift, int num_pages, cudaStream_t stream);
cudaError_t launch_cache_trim(int32_t* table, const int32_t* seqlens, int32_t* refs, int32_t* result, int B,
                              int max_pages, int page_shift, int num_pages, int window, int sink,
                              cudaStream_t stream);
cudaError_t launch_cache_free(int32_t* table, int32_t* seqlens, int32_t* refs, const int32_t* seqs, int32_t* result,
                              int n, int B, int max_pages, int num_pages, cudaStream_t stream);
cudaError_t launch_cache_compact(const int32_t* table, const int32_t* refs, int32_t* table_out, int32_t* refs_out,
                                 int32_t* moves, int32_t* result, int B, int max_pages, int num_pages,
                                 cudaStream_t stream);
cudaError_t launch_cache_copy_pages(void* k, void* v, const int32_t* copies, int n, int num_pages, size_t page_bytes,
                                    cudaStream_t stream);

// Tokens per split and number of splits of the bf16 decode for these sizes.
void decode_split_plan(int B, int Smax, int Hkv, int* split_len, int* nsplit);
// The same for a sliding-window decode (window > 0): splits over the window's span when that
// needs no more splits than the plan for Smax (the workspace is sized by that plan).
void decode_split_plan_window(int B, int Smax, int Hkv, int window, int* split_len, int* nsplit);

// The bf16 decode's workspace, in this order: fp32 partial outputs O [rows, D], fp32 (m, l)
// [rows, 2], then one int split counter per (b, KV head), padded to 16 bytes; rows =
// B * T * Hq * nsplit (T new tokens per sequence). Every entry point that hands the split
// kernel a workspace (caller-provided or the library's own array) lays it out through these.
struct DecodeWorkspace {
  float* o;
  float* ml;
  int* counters;
};
size_t decode_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int nsplit);
DecodeWorkspace decode_workspace_layout(void* base, int B, int T, int Hq, int D, int nsplit);

// fp32 CUDA-core paths (D in {64, 128}).
cudaError_t launch_prefill_f32(const float* q, const float* k, const float* v, const float* lambda, float* out,
                               int B, int S, int Hq, int Hkv, int D, int causal, cudaStream_t stream);
cudaError_t launch_decode_f32(const float* q, const float* kc, const float* vc, const int32_t* seqlens,
                              const float* lambda, float* out, int B, int Smax, int Hq, int Hkv, int D,
                              cudaStream_t stream);

// V1 lambda, broadcast to `rows` rows.
cudaError_t launch_lambda_v1(const float* lq1, const float* lk1, const float* lq2, const float* lk2,
                             float lambda_init, int n_pairs, int d, int rows, float* out, cudaStream_t stream);

// Rotary positions with n_axes axes (rope.cu): q [T,Hq,D] and k [T,Hkv,D] (token strides in
// elements) to q_out and k_out. With block_table the k of every token goes to its row of the
// paged cache k_out [num_pages, 1 << page_shift, Hkv, D], v to v_out; cu_seqlens null: token t is
// sequence t's only new one.
struct RopeParams {
  const void *q, *k, *v;
  void *q_out, *k_out, *v_out;
  long long q_stride, k_stride, v_stride, qo_stride, ko_stride;
  const int32_t* positions;  // [n_axes, T]
  const float* inv_freq;     // [P]
  int sec_end[4];            // first pair past each axis' section
  int n_axes, P, T, Hq, Hkv, D, inverse, interleaved;
  const int32_t *block_table, *seqlens, *cu_seqlens;
  int B, max_pages, page_shift, num_pages;
  int* err;  // debug-bounds build: the device error word
};
cudaError_t launch_rope(const RopeParams& p, bool f32, cudaStream_t stream);

// Address of the device error word on the current device.
cudaError_t device_error_word(int** out);
// The same for kernels that report violated bounds and nothing else (null in the normal build).
inline cudaError_t bounds_error_word(int** out) {
#ifdef DA2_DEBUG_BOUNDS
  return device_error_word(out);
#else
  *out = nullptr;
  return cudaSuccess;
#endif
}

// 4-D bf16 tensor map over a row-major [B,S,H,D] array, box {box0, 1, box2, 1}, 128-byte swizzle.
cudaError_t encode_bshd_bf16(CUtensorMap* map, const void* base, uint64_t D, uint64_t H, uint64_t S, uint64_t B,
                             uint32_t box0, uint32_t box2);

// 4-D bf16 tensor map for the prefill's output stores: [B,S,H,D] (H = Hq/2 pairs), box
// {32, 1, 32, 1} (32 columns of 32 rows of one pair), 64-byte swizzle.
cudaError_t encode_out_bf16(CUtensorMap* map, void* base, uint64_t D, uint64_t H, uint64_t S, uint64_t B);

// V2 lambda projection sigmoid(x W + bias) on tcgen05: tmX over x [T, d_model] bf16 with
// boxes of 64 (d_model) x 128 (tokens), tmW over W [d_model, n_pairs] bf16 with boxes of 64
// (pair columns; those past n_pairs read as zeros) x 64 (d_model), both 128-byte swizzled;
// bias fp32 [n_pairs] or null; d_model % 64 == 0, n_pairs % 8 == 0 and <= 64.
cudaError_t launch_lambda_v2(const CUtensorMap& tmX, const CUtensorMap& tmW, const float* bias, int T, int d_model,
                             int n_pairs, float* out, int* err, cudaStream_t stream);

// 2-D bf16 tensor map over a row-major [rows, cols] array with row stride `row_bytes`, box
// {box_cols, box_rows}, 128-byte swizzle, out-of-range elements read as zero.
cudaError_t encode_2d_bf16(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t row_bytes,
                           uint32_t box_cols, uint32_t box_rows);

}  // namespace da2
