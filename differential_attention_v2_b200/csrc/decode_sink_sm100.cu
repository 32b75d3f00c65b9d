// decode_sink_sm100.cu -- bf16 DiffAttn V2 decode step of a sliding-window layer with sinks: the
// new token of a sequence of n keys sees its last `window` keys and the first `sink` ones,
//   out[b,p] = softmax(q1 K^T/sqrt(D)) V - lambda[b,p] softmax(q2 K^T/sqrt(D)) V
//   over the keys j with j < sink or j >= n - window
// (the window of the "Attention variants" lesson's sliding-window step; the sinks are the few
// first tokens that every query of a trained window layer leans on).
//
// Bound by HBM: each visible K and V row is read once for both branches and all query heads of its
// KV head; with few sequences, by the latency of its dependent steps. The visible keys are two runs,
// cut at multiples of 16 tokens into a list of chunks: those of the sinks, then those of the window.
// Unlike the plain decode, whose span is the whole cache, the list is short (a window), so its parts
// can meet inside the chip:
//
//  * One cluster of up to 16 CTAs per (KV head, sequence); the CTAs take consecutive parts of the
//    list. Each merges its four warps and stores the (max, sum, output) of pair i straight into the
//    shared memory of CTA i % ctas, which joins and writes it after one cluster barrier. No
//    workspace, no counters to clear, one launch. (Reading the others' partials after the barrier
//    cost three dependent trips between SMs and a second barrier before the exit: 2.2 us of 6.3 in
//    a clock trace of one user's step, window 1024.)
//  * A warp is a pipeline of its own: it takes every fourth chunk of its CTA, through a ring of
//    three 8 KB slots that its first lane refills by TMA as soon as the warp has read one. There is
//    no producer warp and no barrier between warps until the merge. A chunk's K (or V), both
//    64-wide halves of d, is one copy of a 5-d tensor map (two where pages hold 8 tokens): with a
//    producer warp issuing the halves of 64 tokens for all, 16 copies of 16-token pages took 0.8 us
//    to issue before the first key could be used.
//  * S^T = K Q^T and O^T += V^T P^T on mma.sync m16n8k16 with the group's heads as N, online softmax
//    per head in between; the score MMAs run as two chains of four.
//  * Rows of a border chunk that the token does not see may hold anything (an unwritten cache
//    row, a page that now belongs to another sequence): their scores are replaced, not scaled,
//    and their V rows are zeroed in shared memory, so no NaN or infinity passes through 0 * V.

#include <atomic>

#include <cooperative_groups.h>

#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace da2 {
namespace decode_sink {

namespace cg = cooperative_groups;

constexpr int HD = 128;
constexpr int kTok = 16;  // tokens per chunk
constexpr int kSlots = 3;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kTileBytes = kTok * HD * 2;      // K or V of a chunk
constexpr uint32_t kSlotBytes = 2 * kTileBytes;
constexpr uint32_t kWarpBytes = kSlots * kSlotBytes;
constexpr uint32_t kOffBar = kWarps * kWarpBytes;
constexpr uint32_t kOffMisc = kOffBar + 8 * kWarps * kSlots;
constexpr int kMaxCluster = 16;
constexpr uint32_t kOffRecv = kOffMisc + 16;       // partials from the cluster's CTAs
constexpr uint32_t kPartBytes = 2 * HD * 4 + 16;   // of one pair from one CTA: O_1, O_2, (m, l) of both
__host__ __device__ inline uint32_t recv_pairs(int pairs, int ctas) {
  return static_cast<uint32_t>((pairs + ctas - 1) / ctas);  // pairs that a CTA joins
}
__host__ __device__ inline uint32_t smem_bytes(int pairs, int ctas) {
  return kOffRecv + recv_pairs(pairs, ctas) * static_cast<uint32_t>(ctas) * kPartBytes + 1024;  // + alignment
}
// of all launches (at most 8 pairs; 8 slots, or one from each of 16 CTAs)
constexpr uint32_t kMaxSmemBytes = kOffRecv + kMaxCluster * kPartBytes + 1024;

struct Params {
  const __nv_bfloat16* q;  // [B,Hq,D]
  const int32_t* seqlens;  // [B]
  const float* lambda;     // [B,Hq/2]
  __nv_bfloat16* out;      // [B,Hq/2,D]
  int* err;
  int Smax, Hq, Hkv, window, sink;
  float scale_log2;
  const int32_t* block_table;  // null: [B,Smax] caches
  int max_pages, page_shift;
};

// The merge buffers of a CTA's warps, over the rings.
template <int NT>
struct Merge {
  float warp_ml[kWarps][8 * NT][2];
  float warp_o[kWarps][8 * NT][HD];
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 2)
decode_sink_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params p) {
  static_assert(sizeof(Merge<NT>) <= kOffBar, "merge buffers");
  pdl_wait();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc);
  cg::cluster_group cl = cg::this_cluster();

  const int ctas = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);
  const int g = blockIdx.y;
  const int b = blockIdx.z;
  const int group = p.Hq / p.Hkv;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // every CTA of the cluster is running once this barrier completes (awaited before the first store
  // to another CTA's shared memory)
  cluster_arrive_relaxed();
  const uint32_t ring = sbase + warp * kWarpBytes, bars = sbase + kOffBar + 8u * kSlots * warp;

  if (lane == 0) {
    if (warp == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      *abort_flag = 0;
    }
    for (int s = 0; s < kSlots; ++s) mbar_init(bars + 8u * s, 1);
    fence_mbar_init();
  }
  // the lambda of the first pair that this warp will write, on its way meanwhile
  const int n_pairs = p.Hq >> 1;
  const size_t pair0 = static_cast<size_t>(b) * n_pairs + g * (group / 2);
  const int my_pair = rank + ctas * warp;
  const float lam0 = my_pair < group / 2 ? *(p.lambda + pair0 + my_pair) : 0.f;

  // visible keys: [0, ns) and [lo, n); chunks 0 .. n_head-1 and from first_w on
  const int n = min(max(*(p.seqlens + b), 0), p.Smax);
  const int lo = max(0, n - p.window);
  const int ns = min(p.sink, lo);
  const int first_w = lo / kTok;
  const int n_head = min((ns + kTok - 1) / kTok, first_w);
  const int total = n_head + (n + kTok - 1) / kTok - first_w;
  // this warp's chunks: c0 + warp, c0 + warp + kWarps, .. < c1
  const int c0 = static_cast<int>(static_cast<long long>(total) * rank / ctas);
  const int c1 = static_cast<int>(static_cast<long long>(total) * (rank + 1) / ctas);
  const int mine = c1 - c0 > warp ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0;
  auto chunk_tok = [&](int k) -> int {
    const int c = c0 + warp + k * kWarps;
    return (c < n_head ? c : first_w + c - n_head) * kTok;
  };
  auto seen = [&](int t) -> bool { return t < ns || (t >= lo && t < n); };
  // some token of [t, t + count) is visible
  auto any_seen = [&](int t, int count) -> bool { return t < ns || (t + count > lo && t < n); };

  // Pages of 8 tokens: two copies of 8 rows, each both halves of d; else one of 16 rows. Row r of a
  // tile is at (r / 8) * sub + half * 64-wide + (r % 8) * 128 bytes.
  const bool small_pages = p.block_table && p.page_shift == 3;
  const uint32_t sub_stride = small_pages ? 2048 : 1024, half_stride = small_pages ? 1024 : 2048;
  // lane l holds the pages of this warp's chunks 32 j + l (entry1: of a chunk's second 8 tokens)
  int entry0 = b, entry1 = b;
  auto load_entries = [&](int k0) {
    if (!p.block_table) return;
    const int k = k0 + lane;
    if (k >= mine) return;
    const int t = chunk_tok(k), lp = t >> p.page_shift;
    const int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_pages;
    if (checked(lp < p.max_pages, p.err)) entry0 = *(row + lp);
    if (small_pages && t + 8 < n && checked(lp + 1 < p.max_pages, p.err)) entry1 = *(row + lp + 1);
  };
  // chunk k into its slot (the whole warp calls; lane 0 copies)
  auto issue = [&](int k) {
    const int e0 = __shfl_sync(0xffffffffu, entry0, k & 31), e1 = __shfl_sync(0xffffffffu, entry1, k & 31);
    if (lane != 0) return;
    const int s = k % kSlots, t = chunk_tok(k);
    const uint32_t bar = bars + 8u * s, dst = ring + s * kSlotBytes;
    const int row = p.block_table ? t & ((1 << p.page_shift) - 1) : t;
    if (!checked(within(dst, kSlotBytes, sbase, kOffBar) && g < p.Hkv, p.err)) return;
    if (!small_pages) {
      mbar_arrive_expect_tx(bar, kSlotBytes);
      tma_load_5d(dst, &tmK, bar, 0, row, 0, g, e0);
      tma_load_5d(dst + kTileBytes, &tmV, bar, 0, row, 0, g, e0);
    } else {
      const bool a = any_seen(t, 8), c = any_seen(t + 8, 8);
      mbar_arrive_expect_tx(bar, (a ? kTileBytes : 0) + (c ? kTileBytes : 0));
      if (a) {
        tma_load_5d(dst, &tmK, bar, 0, row, 0, g, e0);
        tma_load_5d(dst + kTileBytes, &tmV, bar, 0, row, 0, g, e0);
      }
      if (c) {
        tma_load_5d(dst + 2048, &tmK, bar, 0, 0, 0, g, e1);
        tma_load_5d(dst + kTileBytes + 2048, &tmV, bar, 0, 0, 0, g, e1);
      }
    }
  };

  load_entries(0);
  __syncthreads();  // the barriers and the abort flag exist
  int issued = 0;
  for (; issued < kSlots && issued < mine; ++issued) issue(issued);

  // Q^T as B fragments: column n = 8 nt + gl is head n of the group, k = d
  const int gl = lane >> 2;  // fragment row group
  const int tq = lane & 3;   // fragment column pair
  float o[NT][8][4];
  float m_run[NT][2], l_part[NT][2];
  uint32_t qf[NT][8][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = nt * 8 + gl;
    const bool hv = h < group;
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(
        p.q + (static_cast<size_t>(b) * p.Hq + g * group + (hv ? h : 0)) * HD);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      qf[nt][kk][0] = hv ? *(qrow + 8 * kk + tq) : 0u;
      qf[nt][kk][1] = hv ? *(qrow + 8 * kk + tq + 4) : 0u;
    }
    m_run[nt][0] = m_run[nt][1] = -INFINITY;
    l_part[nt][0] = l_part[nt][1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
  }
  // per-lane ldmatrix offsets: K rows lane & 15, 16-byte chunk parity lane >> 4; V as V^T
  const int k_row = lane & 15, k_csel = lane >> 4;
  const int v_row = (lane & 7) + ((lane >> 4) & 1) * 8, v_csel = (lane >> 3) & 1;
  const uint32_t k_off = (k_row >> 3) * sub_stride + (k_row & 7) * 128;
  const uint32_t v_off = (v_row >> 3) * sub_stride + (v_row & 7) * 128;

  for (int k = 0; k < mine; ++k) {
    const int s = k % kSlots;
    // the warp leaves together: the loop body is made of warp-collective instructions
    if (!__all_sync(0xffffffffu, mbar_wait(bars + 8u * s, (k / kSlots) & 1, abort_flag))) break;
    const uint32_t kb = ring + s * kSlotBytes, vb = kb + kTileBytes;
    const int tok = chunk_tok(k);
    const bool edge = !(tok + kTok <= ns || (tok >= lo && tok + kTok <= n));
    if (edge) {
      const int r = lane & 15;
      if (!seen(tok + r)) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          st_shared_v4(vb + (r >> 3) * sub_stride + (lane >> 4) * half_stride + (r & 7) * 128 + 16 * c, 0u, 0u, 0u, 0u);
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
      ldmatrix_x4(kb + k_off + (chunk >> 3) * half_stride + (((chunk & 7) ^ (k_row & 7)) << 4), a0, a1, a2, a3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_m16n8k16_bf16(kk & 1 ? sodd[nt] : sacc[nt], a0, a1, a2, a3, qf[nt][kk][0], qf[nt][kk][1]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) sacc[nt][c] += sodd[nt][c];
    const bool va = !edge || seen(tok + gl), vb8 = !edge || seen(tok + gl + 8);
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
      ldmatrix_x4_trans(vb + v_off + (chunk >> 3) * half_stride + (((chunk & 7) ^ (v_row & 7)) << 4), a0, a1, a2, a3);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_m16n8k16_bf16(o[nt][mt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
    }
    if (edge) fence_proxy_async_shared();  // the zeroed rows come before the next copy into them
    __syncwarp();                          // every lane has read the slot
    if (k + kSlots < mine) {
      if (((k + kSlots) & 31) == 0) load_entries(k + kSlots);
      issue(k + kSlots);
      issued = k + kSlots + 1;
    }
  }
  if (*abort_flag) {
    // every issued copy lands before the shared memory is reused; each wait has its own limit
    for (int k = max(0, issued - kSlots); k < issued; ++k) {
      volatile int none = 0;
      mbar_wait(bars + 8u * (k % kSlots), (k / kSlots) & 1, &none);
    }
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

  // every copy has landed (its warp waited for it): the rings are free for the merge
  __syncthreads();
  Merge<NT>& mg = *reinterpret_cast<Merge<NT>*>(smem);
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
  __syncthreads();
  // Pair i goes to CTA i % ctas, slot i / ctas: [slot][CTA] {O_1[128], O_2[128], m_1, l_1, m_2, l_2}.
  // A CTA whose copies gave up sends l = -1.
  const bool aborted = *abort_flag != 0;
  cluster_wait();
  {
    const int d = threadIdx.x;  // 0..127
#pragma unroll 4
    for (int h = 0; h < group; ++h) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mg.warp_ml[w][h][0]);
      const float Mu = (M == -INFINITY) ? 0.f : M;
      float O = 0.f, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float sc = fast_exp2(mg.warp_ml[w][h][0] - Mu);
        O += mg.warp_o[w][h][d] * sc;
        L += mg.warp_ml[w][h][1] * sc;
      }
      const int i = h >> 1, br = h & 1;
      const uint32_t at = kOffRecv + (static_cast<uint32_t>(i / ctas) * ctas + rank) * kPartBytes;
      if (!checked(i / ctas < static_cast<int>(recv_pairs(group / 2, ctas)), p.err)) continue;
      float* dst = reinterpret_cast<float*>(cl.map_shared_rank(smem + at, i % ctas));
      dst[br * HD + d] = O;
      if (d == 0) *reinterpret_cast<float2*>(dst + 2 * HD + 2 * br) = make_float2(M, aborted ? -1.f : L);
    }
  }
  cl.sync();  // every partial has arrived; nothing is stored to another CTA after this

  // a warp joins a pair: a lane takes 4 of d, and lane r < ctas the (max, sum) of CTA r's partials
  for (int i = my_pair; i < group / 2; i += ctas * kWarps) {
    const uint8_t* part = smem + kOffRecv + static_cast<uint32_t>(i / ctas) * ctas * kPartBytes;
    float4 ml = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    if (lane < ctas) ml = *reinterpret_cast<const float4*>(part + lane * kPartBytes + 2 * HD * 4);
    if (__any_sync(0xffffffffu, ml.y < 0.f || ml.w < 0.f)) {
      if (lane == 0) atomicCAS(p.err, 0, kErrDecodeWait);
      continue;
    }
    float res[2][4];
#pragma unroll
    for (int br = 0; br < 2; ++br) {
      const float m = br ? ml.z : ml.x, l = br ? ml.w : ml.y;
      float M = m;
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      const float sc = fast_exp2(m - ((M == -INFINITY) ? 0.f : M));
      float L = l * sc;
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int r = 0; r < ctas; ++r) {
        const float w = __shfl_sync(0xffffffffu, sc, r);
        const float4 v = reinterpret_cast<const float4*>(part + r * kPartBytes + br * HD * 4)[lane];
        acc.x += v.x * w;
        acc.y += v.y * w;
        acc.z += v.z * w;
        acc.w += v.w * w;
      }
      L = __shfl_sync(0xffffffffu, L, 0);
      const float inv = (L > 0.f) ? 1.f / L : 0.f;  // an empty sequence: zeros
      res[br][0] = __fmul_rn(acc.x, inv);
      res[br][1] = __fmul_rn(acc.y, inv);
      res[br][2] = __fmul_rn(acc.z, inv);
      res[br][3] = __fmul_rn(acc.w, inv);
    }
    const size_t row = pair0 + i;
    const float lam = i == my_pair ? lam0 : *(p.lambda + row);
    uint2 packed;
    packed.x = pack_bf16x2(__fmaf_rn(-lam, res[1][0], res[0][0]), __fmaf_rn(-lam, res[1][1], res[0][1]));
    packed.y = pack_bf16x2(__fmaf_rn(-lam, res[1][2], res[0][2]), __fmaf_rn(-lam, res[1][3], res[0][3]));
    if (checked(row < static_cast<size_t>(gridDim.z) * n_pairs, p.err))
      reinterpret_cast<uint2*>(p.out + row * HD)[lane] = packed;
  }
}

// CTAs per (KV head, sequence): as many as fit the GPU at two CTAs per SM, but no more than there are
// groups of 64 keys. 16 (a non-portable size whose receive buffers leave one CTA per SM) only where all
// clusters of it are resident together: it needs 16 SMs of one GPC, which 7 clusters at a time found on
// the B200 measured here. us in a graph, 4 sinks, groups of 8; CTAs per cluster 1 / 2 / 4 / 8 / 16:
//   units (KV heads x sequences)  window
//   1      1024    14.6  10.0   7.6   6.5   6.2      7      1024       .     .   7.7   6.6   6.3
//   1      8192    79.4  42.1  23.3  14.3  10.0      7      8192       .     .  23.6  14.5  10.4
//   1     32768     300   153    79  42.4  24.1      7     32768       .     .    82  43.6  25.9
//   8      1024    14.7  10.0   7.8   6.5  10.6      8     32768     306   156    81  43.7  48.5
//   32     1024    15.0  10.1   8.1   7.9  27.8      64     4096    44.2  27.1  26.6  31.3  69.7
//   128    1024    16.9  16.2  21.6  29.7  99.2      256    1024    27.3  31.4  39.7  56.3   200
int cluster_size(long long units, int span, int resident16) {
  int c = 1;
  while (c < 8 && 2 * c * units <= 296 && span > c) c *= 2;
  return c == 8 && span > 8 && units <= resident16 ? 16 : c;
}

// How many clusters of 16 the current device runs at a time (GPUs differ in the SMs of their GPCs);
// asked once per device and kernel.
template <int NT>
cudaError_t resident_clusters_of_16(int* n) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // 1 + the number, 0: not asked yet
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  if (device < kDevices && known[device] > 0) {
    *n = known[device] - 1;
    return cudaSuccess;
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kMaxCluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kMaxCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMaxSmemBytes;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(n, decode_sink_kernel<NT>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    *n = 0;  // a device without such clusters: 8 CTAs do
  }
  if (device < kDevices) known[device] = 1 + *n;
  return cudaSuccess;
}

}  // namespace decode_sink

cudaError_t launch_decode_sink(const CUtensorMap& tmK, const CUtensorMap& tmV, const __nv_bfloat16* q,
                               const int32_t* seqlens, const float* lambda, __nv_bfloat16* out, int* err, int B,
                               int Smax, int Hq, int Hkv, int window, int sink, const int32_t* block_table,
                               int max_pages, int page_shift, cudaStream_t stream) {
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
  // most groups of 64 keys that a sequence can have
  const long long keys = static_cast<long long>(window) + sink;
  const int span = static_cast<int>((keys < Smax ? keys : Smax) / 64) + 1;
  const bool wide = Hq / Hkv > 8;
  auto kernel = wide ? decode_sink_kernel<2> : decode_sink_kernel<1>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmemBytes);
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>(B) * Hkv;
  int resident16 = 0;
  if (units <= 148 / kMaxCluster) {  // (more cannot be resident at one CTA per SM)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    e = wide ? resident_clusters_of_16<2>(&resident16) : resident_clusters_of_16<1>(&resident16);
    if (e != cudaSuccess) return e;
  }
  const int c = cluster_size(units, span, resident16);
  const uint32_t smem = smem_bytes(Hq / Hkv / 2, c);
  return launch_chained(kernel, dim3(static_cast<unsigned>(c), static_cast<unsigned>(Hkv), static_cast<unsigned>(B)),
                        dim3(kThreads), smem, c, stream, tmK, tmV, p);
}

}  // namespace da2
