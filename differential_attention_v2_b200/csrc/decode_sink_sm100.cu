// decode_sink_sm100.cu -- bf16 DiffAttn V2 decode step of a sliding-window layer with sinks: the
// new token of a sequence of n keys sees its last `window` keys and the first `sink` ones,
//   out[b,p] = softmax(q1 K^T/sqrt(D)) V - lambda[b,p] softmax(q2 K^T/sqrt(D)) V
//   over the keys j with j < sink or j >= n - window
// (the window of the "Attention variants" lesson's sliding-window step; the sinks are the few
// first tokens that every query of a trained window layer leans on).
//
// Bound by HBM: each visible K and V row is read once for both branches and all query heads of its
// KV head. The visible keys are two runs, cut at multiples of 64 tokens into a list of stages:
// those of the sinks, then those of the window. Unlike the plain decode, whose span is the whole
// cache, the list is short (a window), so its splits can meet inside the chip:
//
//  * One cluster of up to 16 CTAs per (KV head, sequence); the CTAs take consecutive parts of the
//    list. Each merges its four warps in shared memory, and after a cluster barrier the CTAs read
//    one another's (max, sum, output) through distributed shared memory and write the pairs. No
//    workspace, no counters to clear, one launch.
//  * A producer warp fills a 3-stage ring by TMA (64 tokens of K and V, 128-byte swizzle). Its
//    lanes hold the next pages' table entries, and each lane issues the copies of its own page.
//    Stages at a border of a run copy only the 8-token groups that hold a visible key: four
//    sinks cost 4 KB, not 32.
//  * Four consumer warps take 16 tokens of every stage: S^T = K Q^T and O^T += V^T P^T on
//    mma.sync m16n8k16 with the group's heads as N, online softmax per head in between.
//  * Rows of a border stage that the token does not see may hold anything (an unwritten cache
//    row, a page that now belongs to another sequence): their scores are replaced, not scaled,
//    and their V rows are zeroed in shared memory, so no NaN or infinity passes through 0 * V.

#include <cooperative_groups.h>

#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace da2 {
namespace decode_sink {

namespace cg = cooperative_groups;

constexpr int HD = 128;
constexpr int kTok = 64;  // tokens per stage
constexpr int kEdge = 8;  // tokens per copy of a border stage: one swizzle atom of rows
constexpr int kStages = 3;
constexpr int kConsumerWarps = 4;
constexpr int kThreads = 32 * (kConsumerWarps + 1);
constexpr uint32_t kHalfBytes = kTok * 64 * 2;    // 64 tokens x 64 d bf16
constexpr uint32_t kStageBytes = 4 * kHalfBytes;  // K lo/hi, V lo/hi
constexpr uint32_t kOffBar = kStages * kStageBytes;
constexpr uint32_t kOffMisc = kOffBar + 8 * 2 * kStages;
constexpr uint32_t kSmemUsed = kOffMisc + 16;
constexpr uint32_t kSmemBytes = kSmemUsed + 1024;  // slack for the 1024-byte alignment
constexpr int kMaxCluster = 16;

struct Params {
  const __nv_bfloat16* q;  // [B,Hq,D]
  const int32_t* seqlens;  // [B]
  const float* lambda;     // [B,Hq/2]
  __nv_bfloat16* out;      // [B,Hq/2,D]
  int* err;
  int Smax, Hq, Hkv, window, sink;
  float scale_log2;
  const int32_t* block_table;  // null: [B,Smax] caches
  int max_pages, page_shift, box_tok;
};

// The part of the merge buffers that other CTAs read, at the front of the ring.
template <int NT>
struct Merge {
  float ml[8 * NT][2];
  float o[8 * NT][HD];
  float warp_ml[kConsumerWarps][8 * NT][2];
  float warp_o[kConsumerWarps][8 * NT][HD];
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 2)
decode_sink_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ CUtensorMap tmK8, const __grid_constant__ CUtensorMap tmV8,
                   const Params p) {
  static_assert(sizeof(Merge<NT>) <= kOffBar, "merge buffers");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto full = [&](int s) -> uint32_t { return sbase + kOffBar + 8u * s; };
  auto empty = [&](int s) -> uint32_t { return sbase + kOffBar + 8u * (kStages + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc);
  cg::cluster_group cl = cg::this_cluster();

  const int ctas = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);
  const int g = blockIdx.y;
  const int b = blockIdx.z;
  const int group = p.Hq / p.Hkv;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 32 * kConsumerWarps) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmK8);
    tma_prefetch_desc(&tmV8);
  }
  // the lambda of the first pair that this warp will write, on its way meanwhile
  const int n_pairs = p.Hq >> 1;
  const size_t pair0 = static_cast<size_t>(b) * n_pairs + g * (group / 2);
  const int my_pair = rank + ctas * warp;
  const float lam0 = my_pair < group / 2 ? __ldg(p.lambda + pair0 + my_pair) : 0.f;

  // visible keys: [0, ns) and [lo, n); stages 0 .. n_head-1 and from first_w on
  const int n = min(max(__ldg(p.seqlens + b), 0), p.Smax);
  const int lo = max(0, n - p.window);
  const int ns = min(p.sink, lo);
  const int first_w = lo / kTok;
  const int n_head = min((ns + kTok - 1) / kTok, first_w);
  const int total = n_head + (n + kTok - 1) / kTok - first_w;
  const int i0 = static_cast<int>(static_cast<long long>(total) * rank / ctas);
  const int i1 = static_cast<int>(static_cast<long long>(total) * (rank + 1) / ctas);
  auto stage_tok = [&](int i) -> int { return (i < n_head ? i : first_w + i - n_head) * kTok; };
  // every token of the stage is visible
  auto whole = [&](int tok) -> bool { return tok + kTok <= ns || (tok >= lo && tok + kTok <= n); };
  auto seen = [&](int t) -> bool { return t < ns || (t >= lo && t < n); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kConsumerWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

  const int gl = lane >> 2;  // fragment row group
  const int tq = lane & 3;   // fragment column pair
  float o[NT][8][4];
  float m_run[NT][2], l_part[NT][2];

  if (warp == kConsumerWarps) {
    // --------------------------------------------------------------------- producer
    // Lane 8 u + c serves group c of stages i with (i - i0) % 4 == u: the entry of its page is
    // loaded four stages ahead. Whole stages use 64 / box_tok groups, border stages eight.
    auto entry = [&](int i) -> int {
      if (i >= i1 || !p.block_table) return b;
      const int tok = stage_tok(i), sub = whole(tok) ? p.box_tok : kEdge;
      const int t = tok + (lane & 7) * sub;
      if ((lane & 7) * sub >= kTok || t >= n) return -1;
      const int lp = t >> p.page_shift;
      return checked(lp < p.max_pages, p.err) ? __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + lp) : -1;
    };
    int next = entry(i0 + (lane >> 3));
    int issued = i0;
    bool ok = true;
    for (int i = i0; i < i1 && ok; ++i) {
      const int k = i - i0, s = k % kStages;
      ok = __all_sync(0xffffffffu, mbar_wait(empty(s), ((k / kStages) & 1) ^ 1, abort_flag));
      if (!ok) break;
      const int tok = stage_tok(i);
      const bool all = whole(tok);
      const int sub = all ? p.box_tok : kEdge;
      // this lane's group of the stage, and whether any of its tokens is visible
      const int at = (lane & 7) * sub, t = tok + at;
      const bool mine = (lane >> 3) == (k & 3) && at < kTok &&
                        (all || t < ns || (t + kEdge > lo && t < n));
      const unsigned groups = __ballot_sync(0xffffffffu, mine);
      const uint32_t dst = sbase + s * kStageBytes;
      if (lane == 0) mbar_arrive_expect_tx(full(s), static_cast<uint32_t>(__popc(groups)) * sub * 512u);
      __syncwarp();
      if (mine && checked(within(dst, kStageBytes, sbase, kOffBar) && g < p.Hkv, p.err)) {
        const CUtensorMap* mk = all ? &tmK : &tmK8;
        const CUtensorMap* mv = all ? &tmV : &tmV8;
        const int row = p.block_table ? t & ((1 << p.page_shift) - 1) : t;
        const uint32_t d = dst + static_cast<uint32_t>(at) * 128u;
        tma_load_4d(d + 0 * kHalfBytes, mk, full(s), 0, g, row, next);
        tma_load_4d(d + 1 * kHalfBytes, mk, full(s), 64, g, row, next);
        tma_load_4d(d + 2 * kHalfBytes, mv, full(s), 0, g, row, next);
        tma_load_4d(d + 3 * kHalfBytes, mv, full(s), 64, g, row, next);
      }
      __syncwarp();
      if ((lane >> 3) == (k & 3)) next = entry(i + 4);
      issued = i + 1;
    }
    if (*abort_flag) {
      // every issued copy lands before the shared memory is reused; each wait has its own limit
      for (int i = max(i0, issued - kStages); i < issued; ++i) {
        volatile int none = 0;
        mbar_wait(full((i - i0) % kStages), ((i - i0) / kStages) & 1, &none);
      }
    }
  } else {
    // -------------------------------------------------------------------- consumers
    // Q^T as B fragments: column n = 8 nt + gl is head n of the group, k = d
    uint32_t qf[NT][8][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + gl;
      const bool hv = h < group;
      const uint32_t* qrow = reinterpret_cast<const uint32_t*>(
          p.q + (static_cast<size_t>(b) * p.Hq + g * group + (hv ? h : 0)) * HD);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        qf[nt][kk][0] = hv ? __ldg(qrow + 8 * kk + tq) : 0u;
        qf[nt][kk][1] = hv ? __ldg(qrow + 8 * kk + tq + 4) : 0u;
      }
      m_run[nt][0] = m_run[nt][1] = -INFINITY;
      l_part[nt][0] = l_part[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
    }
    // per-lane ldmatrix row and chunk selectors
    const int k_row = 16 * warp + (lane & 15);
    const int k_csel = (lane >> 4) & 1;
    const int v_row = 16 * warp + (lane & 7) + ((lane >> 4) & 1) * 8;
    const int v_csel = (lane >> 3) & 1;

    for (int i = i0; i < i1; ++i) {
      const int k = i - i0, s = k % kStages;
      // the warp leaves together: the loop body is made of warp-collective instructions
      if (!__all_sync(0xffffffffu, mbar_wait(full(s), (k / kStages) & 1, abort_flag))) break;
      const uint32_t kb = sbase + s * kStageBytes, vb = kb + 2 * kHalfBytes;
      const int tok = stage_tok(i);
      const bool edge = !whole(tok);
      if (edge) {
        const int r = 16 * warp + (lane & 15);
        if (!seen(tok + r)) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            st_shared_v4(vb + (lane >> 4) * kHalfBytes + r * 128 + 16 * c, 0u, 0u, 0u, 0u);
        }
        __syncwarp();
      }
      // two accumulators (even and odd K-steps): half the length of the chain of dependent MMAs
      float sacc[NT][4], sodd[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) sacc[nt][c] = sodd[nt][c] = 0.f;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int chunk = 2 * kk + k_csel;
        uint32_t a0, a1, a2, a3;
        ldmatrix_x4(kb + (chunk >> 3) * kHalfBytes + k_row * 128 + (((chunk & 7) ^ (k_row & 7)) << 4), a0, a1, a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_m16n8k16_bf16(kk & 1 ? sodd[nt] : sacc[nt], a0, a1, a2, a3, qf[nt][kk][0], qf[nt][kk][1]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) sacc[nt][c] += sodd[nt][c];
      const int ta = tok + 16 * warp + gl;
      const bool va = !edge || seen(ta), vb8 = !edge || seen(ta + 8);
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[4], pr[4];
        x[0] = va ? sacc[nt][0] * p.scale_log2 : -INFINITY;
        x[1] = va ? sacc[nt][1] * p.scale_log2 : -INFINITY;
        x[2] = vb8 ? sacc[nt][2] * p.scale_log2 : -INFINITY;
        x[3] = vb8 ? sacc[nt][3] * p.scale_log2 : -INFINITY;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(x[c], x[c + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float m_new = fmaxf(m_run[nt][c], mx);
          const float m_use = (m_new == -INFINITY) ? 0.f : m_new;  // nothing visible yet
          const float alpha = fast_exp2(m_run[nt][c] - m_use);
          m_run[nt][c] = m_new;
          pr[c] = fast_exp2(x[c] - m_use);
          pr[c + 2] = fast_exp2(x[c + 2] - m_use);
          l_part[nt][c] = l_part[nt][c] * alpha + pr[c] + pr[c + 2];
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            o[nt][mt][c] *= alpha;
            o[nt][mt][c + 2] *= alpha;
          }
        }
        // P^T fragments: the two 8x8 (token x head) blocks transposed
        pb[nt][0] = movmatrix_trans(pack_bf16x2(pr[0], pr[1]));
        pb[nt][1] = movmatrix_trans(pack_bf16x2(pr[2], pr[3]));
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        const int chunk = 2 * mt + v_csel;
        uint32_t a0, a1, a2, a3;
        ldmatrix_x4_trans(vb + (chunk >> 3) * kHalfBytes + v_row * 128 + (((chunk & 7) ^ (v_row & 7)) << 4), a0, a1, a2,
                          a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_m16n8k16_bf16(o[nt][mt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
      if (edge) fence_proxy_async_shared();  // the zeroed rows come before the next copy into them
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = l_part[nt][c];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        l_part[nt][c] = v;
      }
  }

  // every copy has landed (consumers waited on each full barrier): the ring is free for the merge
  __syncthreads();
  Merge<NT>& mg = *reinterpret_cast<Merge<NT>*>(smem);
  if (warp < kConsumerWarps) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          mg.warp_o[warp][nt * 8 + 2 * tq + (c & 1)][16 * mt + gl + (c >> 1) * 8] = o[nt][mt][c];
      if (gl == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mg.warp_ml[warp][nt * 8 + 2 * tq + c][0] = m_run[nt][c];
          mg.warp_ml[warp][nt * 8 + 2 * tq + c][1] = l_part[nt][c];
        }
      }
    }
  }
  __syncthreads();
  if (warp < kConsumerWarps) {
    const int d = threadIdx.x;  // 0..127
    for (int h = 0; h < group; ++h) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, mg.warp_ml[w][h][0]);
      const float Mu = (M == -INFINITY) ? 0.f : M;
      float O = 0.f, L = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumerWarps; ++w) {
        const float sc = fast_exp2(mg.warp_ml[w][h][0] - Mu);
        O += mg.warp_o[w][h][d] * sc;
        L += mg.warp_ml[w][h][1] * sc;
      }
      mg.o[h][d] = O;
      if (d == 0) {
        mg.ml[h][0] = M;
        mg.ml[h][1] = L;
      }
    }
  }
  cl.sync();

  // Pair i of the group goes to warp (i / ctas) of CTA i % ctas; a lane takes 4 of d.
  bool aborted = false;
  for (int r = 0; r < ctas; ++r) aborted |= *cl.map_shared_rank(const_cast<int*>(abort_flag), r) != 0;
  if (aborted) {
    if (threadIdx.x == 0) atomicCAS(p.err, 0, kErrDecodeWait);
  } else {
    for (int i = my_pair; i < group / 2; i += ctas * (kConsumerWarps + 1)) {
      float res[2][4];
#pragma unroll
      for (int br = 0; br < 2; ++br) {
        const int h = 2 * i + br;
        float M = -INFINITY, L = 0.f;
        for (int r = 0; r < ctas; ++r) M = fmaxf(M, cl.map_shared_rank(&mg, r)->ml[h][0]);
        const float Mu = (M == -INFINITY) ? 0.f : M;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < ctas; ++r) {
          const Merge<NT>* m = cl.map_shared_rank(&mg, r);
          const float sc = fast_exp2(m->ml[h][0] - Mu);
          L += m->ml[h][1] * sc;
          const float4 v = reinterpret_cast<const float4*>(m->o[h])[lane];
          acc.x += v.x * sc;
          acc.y += v.y * sc;
          acc.z += v.z * sc;
          acc.w += v.w * sc;
        }
        const float inv = (L > 0.f) ? 1.f / L : 0.f;  // an empty sequence: zeros
        res[br][0] = __fmul_rn(acc.x, inv);
        res[br][1] = __fmul_rn(acc.y, inv);
        res[br][2] = __fmul_rn(acc.z, inv);
        res[br][3] = __fmul_rn(acc.w, inv);
      }
      const size_t row = pair0 + i;
      const float lam = i == my_pair ? lam0 : __ldg(p.lambda + row);
      uint2 packed;
      packed.x = pack_bf16x2(__fmaf_rn(-lam, res[1][0], res[0][0]), __fmaf_rn(-lam, res[1][1], res[0][1]));
      packed.y = pack_bf16x2(__fmaf_rn(-lam, res[1][2], res[0][2]), __fmaf_rn(-lam, res[1][3], res[0][3]));
      if (checked(row < static_cast<size_t>(gridDim.z) * n_pairs, p.err))
        reinterpret_cast<uint2*>(p.out + row * HD)[lane] = packed;
    }
  }
  cl.sync();  // no CTA leaves while another reads its partial
}

// CTAs per (KV head, sequence): as many as fit the GPU at two CTAs per SM, but no more than there
// are stages; 16 (a non-portable size, slow to place) only for long lists. Measured on B200 (us, 8
// KV heads, 4 sinks; CTAs per cluster 1 / 2 / 4 / 8 / 16):
//   B=1,  window 1024    16.6  11.3   8.6   7.7   8.8
//   B=1,  window 32768    316   161    84    46    31
//   B=8,  window 4096    45.6  27.9  26.6  32.5  56.3
//   B=32, window 1024    28.5  33.4  45.4  71.4   162
int cluster_size(long long units, int span) {
  int c = 1;
  while (c < kMaxCluster && 2 * c * units <= 296 && span > c && (c < 8 || span >= 256)) c *= 2;
  return c;
}

}  // namespace decode_sink

cudaError_t launch_decode_sink(const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmK8,
                               const CUtensorMap& tmV8, const __nv_bfloat16* q, const int32_t* seqlens,
                               const float* lambda, __nv_bfloat16* out, int* err, int B, int Smax, int Hq, int Hkv,
                               int window, int sink, const int32_t* block_table, int max_pages, int page_shift,
                               cudaStream_t stream) {
  using namespace decode_sink;
  Params p;
  p.q = q;
  p.seqlens = seqlens;
  p.lambda = lambda;
  p.out = out;
  p.err = err;
  p.Smax = Smax;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.window = window;
  p.sink = sink;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(HD));
  p.block_table = block_table;
  p.max_pages = max_pages;
  p.page_shift = page_shift;
  p.box_tok = block_table ? min(1 << page_shift, kTok) : kTok;
  // most stages that a sequence can have
  const long long keys = static_cast<long long>(window) + sink;
  const int span = static_cast<int>((keys < Smax ? keys : Smax) / kTok) + 1;
  const int c = cluster_size(static_cast<long long>(B) * Hkv, span);
  auto kernel = Hq / Hkv > 8 ? decode_sink_kernel<2> : decode_sink_kernel<1>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  if (c > 8) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(c);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(c), static_cast<unsigned>(Hkv), static_cast<unsigned>(B));
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, tmK, tmV, tmK8, tmV8, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace da2
