// rope.cu -- rotary positions with several axes on q and k, alone or fused with the write of the
// new tokens' k and v into a paged cache.
//
// Both heads of a DiffAttn pair and their shared keys carry positions as rotations: dimensions
// (a, b) of pair c of token t turn by the angle
//     phi[t, c] = positions[axis(c), t] * inv_freq[c],      (a, b) -> (a cos - b sin, b cos + a sin)
// where the frequency pairs 0 .. P-1 are dealt to the axes in consecutive sections (time, height,
// width for images and video; one section is plain rotary). Pairs are dimensions (c, c + P), or
// (2c, 2c+1) when interleaved; dimensions from 2P on pass through. The rotation is orthogonal, so
// its gradient is the rotation by -phi (`inverse`).
//
// Bound by HBM: every element is read and written once, 3 flops each. A warp takes one token and a
// run of its heads, and no thread waits for another: a lane owns the same N pairs of every head it
// visits, so their cos and sin stay in registers (the lanes that own the same pairs of different
// heads compute a share each and exchange them). Memory is kept busy by the number of warps: one
// head per lane in flight at 40 warps an SM measured 97 us for 16,384 tokens of 64 + 8 bf16 heads
// of 128 (604 MB, 6.23 TB/s, 0.96 of a plain copy), two heads at 32 warps 99.6, and a CTA per
// token with the angles in shared memory 158 (it issued three times the instructions, and its
// warps waited for one another). Append holds more addresses and runs 32 warps: 60 us for 8,192
// tokens (336 MB, 5.6 TB/s). The angle is formed in 64 bits (an integer position times a fp32 frequency needs up to
// 55 bits; at position 1e5 a fp32 product is off by 1e-2 radians), reduced to a fraction of a turn
// there, and only then rounded to fp32 for sincospif.
//
// Append: k goes to the row of its page (token i of sequence b's n_b new ones is logical position
// seqlens[b] - n_b + i) and v beside it, so that neither is written to a buffer in between.

#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace da2 {
namespace rope {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

// The N elements of a vector in fp32, and back with one rounding.
template <int N>
__device__ __forceinline__ void unpack(const Vec<float, N>& a, float (&f)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = a.v[e];
}
template <int N>
__device__ __forceinline__ void pack(const float (&f)[N], Vec<float, N>& a) {
#pragma unroll
  for (int e = 0; e < N; ++e) a.v[e] = f[e];
}
template <int N>
__device__ __forceinline__ void unpack(const Vec<__nv_bfloat16, N>& a, float (&f)[N]) {
  if constexpr (N == 1) {
    f[0] = __bfloat162float(a.v[0]);
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&a);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
}
template <int N>
__device__ __forceinline__ void pack(const float (&f)[N], Vec<__nv_bfloat16, N>& a) {
  if constexpr (N == 1) {
    a.v[0] = __float2bfloat16_rn(f[0]);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&a);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
  }
}

// Logical position -> row of the paged cache for token t; -1: not stored, -2: not a token.
__device__ __forceinline__ long long cache_row(const RopeParams& p, int t, int lane) {
  int b = t, end = t + 1;
  if (p.cu_seqlens) {
    b = -1;
    for (int b0 = 0; b0 < p.B && b < 0; b0 += 32) {
      const int i = b0 + lane;
      const bool in = i < p.B && *(p.cu_seqlens + i) <= t && t < *(p.cu_seqlens + i + 1);
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (m) b = b0 + __ffs(m) - 1;
    }
    if (b < 0) return -2;  // behind the last sequence
    end = *(p.cu_seqlens + b + 1);
  }
  const int at = *(p.seqlens + b) - (end - t);
  if (at < 0 || (at >> p.page_shift) >= p.max_pages) return -1;
  if (!checked(b < p.B, p.err)) return -1;
  const int page = *(p.block_table + static_cast<size_t>(b) * p.max_pages + (at >> p.page_shift));
  if (page < 0 || page >= p.num_pages) return -1;
  return (static_cast<long long>(page) << p.page_shift) + (at & ((1 << p.page_shift) - 1));
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Heads h, h + step, .. < n of one tensor (of `heads`) at element offsets off + h * D: turned, or copied.
template <typename T, int N, bool kInter, bool kTurn>
__device__ __forceinline__ void walk(const T* src, T* dst, int h, int step, int n, int heads, int D,
                                     int ra, int rb, const float (&co)[N], const float (&si)[N], int* err) {
  using V = Vec<T, N>;
  for (; h < n; h += step) {
    if (!checked(h >= 0 && h < heads && ra + N <= D && rb + N <= D, err)) continue;
    V x = *reinterpret_cast<const V*>(src + h * D + ra);
    V y = *reinterpret_cast<const V*>(src + h * D + rb);
    if constexpr (kTurn) {
      float a[N], b[N];
      unpack(x, a);
      unpack(y, b);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        // pair e of the unit: (a[e], b[e]), or neighbours when interleaved
        float& fa = kInter ? (2 * e < N ? a[(2 * e) % N] : b[(2 * e) % N]) : a[e];
        float& fb = kInter ? (2 * e + 1 < N ? a[(2 * e + 1) % N] : b[(2 * e + 1) % N]) : b[e];
        const float u = fa * co[e] - fb * si[e];
        fb = fb * co[e] + fa * si[e];
        fa = u;
      }
      pack(a, x);
      pack(b, y);
    }
    *reinterpret_cast<V*>(dst + h * D + ra) = x;
    *reinterpret_cast<V*>(dst + h * D + rb) = y;
  }
}

// Lane l works on unit r = l % per_head of head l / per_head of each step, per_head = min(units
// per head, 32). A unit is N pairs of a head (two vectors of N elements), or 2N of its dimensions
// that pass through: units 0 .. P/N-1 rotate, the rest and all of a v head are copied.
template <typename T, int N, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kThreads, kAppend ? 8 : 10)
rope_kernel(const RopeParams p, const int chunks, const int chunk_heads) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(item / chunks);
  if (t >= p.T) return;  // the whole warp
  const int uph = p.D / (2 * N), upr = p.P / N;
  const int per_head = min(uph, 32), hpw = 32 / per_head;
  const int heads = p.Hq + p.Hkv * (kAppend ? 2 : 1);
  const int h0 = static_cast<int>(item - static_cast<long long>(t) * chunks) * chunk_heads;
  const int h1 = min(heads, h0 + chunk_heads);
  const int hs = lane / per_head;  // hpw: this lane has no head (32 is not a multiple of per_head)
  const size_t tt = static_cast<size_t>(t);

  const T* q = static_cast<const T*>(p.q) + tt * p.q_stride;
  // this lane's first head on its way to L2 while the angles are computed
  if (h0 + hs < p.Hq) prefetch_l2(q + static_cast<size_t>(h0 + hs) * p.D + (lane % per_head) * N);
  const long long row = kAppend ? cache_row(p, t, lane) : 0;
  if (kAppend && row == -2) return;

  for (int r0 = 0; r0 < uph; r0 += per_head) {
    const int r = r0 + lane % per_head;
    const bool rot = r < upr;
    // cos and sin of the unit's pairs: in round j lane hs of a unit computes pair j * hpw + hs, and
    // the unit's lanes exchange them
    float co[N], si[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      co[e] = 1.f;
      si[e] = 0.f;
    }
#pragma unroll 1
    for (int j = 0; j * hpw < N; ++j) {
      const int e0 = j * hpw + hs, c = r * N + e0;
      float s = 0.f, k = 1.f;
      if (rot && e0 < N && checked(c < p.P, p.err)) {
        int axis = 0;
        while (axis + 1 < p.n_axes && c >= p.sec_end[axis]) ++axis;
        double turn = static_cast<double>(*(p.positions + static_cast<size_t>(axis) * p.T + t)) *
                      static_cast<double>(*(p.inv_freq + c)) * 0.15915494309189535;
        turn -= rint(turn);
        sincospif(static_cast<float>(2.0 * turn), &s, &k);
        if (p.inverse) s = -s;
      }
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e >= j * hpw && e < (j + 1) * hpw) {
          const int from = (e - j * hpw) * per_head + lane % per_head;
          co[e] = __shfl_sync(0xffffffffu, k, from);
          si[e] = __shfl_sync(0xffffffffu, s, from);
        }
    }
    const int ca = 2 * N * r, cb = ca + N;  // offsets of a unit that is copied
    const int ra = rot && !kInter ? r * N : ca, rb = rot && !kInter ? p.P + r * N : cb;
    const bool mine = hs < hpw && r < uph;
    if (!mine) continue;
    // this lane's heads of q, then k, then v among h0 + hs, h0 + hs + hpw, .. < h1
    T* qo = static_cast<T*>(p.q_out) + tt * p.qo_stride;
    const int nq = min(h1, p.Hq);
    int h = h0 + hs;
    // a unit that passes through has cos 1 and sin 0, but is copied: -0 and NaN keep their bits
    if (rot) walk<T, N, kInter, true>(q, qo, h, hpw, nq, p.Hq, p.D, ra, rb, co, si, p.err);
    else walk<T, N, kInter, false>(q, qo, h, hpw, nq, p.Hq, p.D, ra, rb, co, si, p.err);
    if (h < p.Hq) h += (p.Hq - h + hpw - 1) / hpw * hpw;
    if (h >= h1 || (kAppend && row < 0)) continue;  // (no page for this token: only its q is written)
    const size_t at = kAppend ? static_cast<size_t>(row) * p.Hkv * p.D : tt * p.ko_stride;
    const T* k = static_cast<const T*>(p.k) + tt * p.k_stride;
    T* ko = static_cast<T*>(p.k_out) + at;
    const int nk = min(h1 - p.Hq, p.Hkv);
    if (rot) walk<T, N, kInter, true>(k, ko, h - p.Hq, hpw, nk, p.Hkv, p.D, ra, rb, co, si, p.err);
    else walk<T, N, kInter, false>(k, ko, h - p.Hq, hpw, nk, p.Hkv, p.D, ra, rb, co, si, p.err);
    if (kAppend) {
      h -= p.Hq + p.Hkv;
      if (h < 0) h += (-h + hpw - 1) / hpw * hpw;
      walk<T, N, kInter, false>(static_cast<const T*>(p.v) + tt * p.v_stride, static_cast<T*>(p.v_out) + at, h, hpw,
                                h1 - p.Hq - p.Hkv, p.Hkv, p.D, ca, cb, co, si, p.err);
    }
  }
}

template <typename T, int N>
cudaError_t launch_n(const RopeParams& p, cudaStream_t stream) {
  const bool append = p.block_table != nullptr;
  const int uph = p.D / (2 * N), hpw = 32 / (uph < 32 ? uph : 32);
  const int heads = p.Hq + p.Hkv * (append ? 2 : 1);
  // One warp per token; with few tokens (decode steps) a token's heads are dealt to several warps,
  // down to four heads per lane, until there are 8 warps for every SM.
  const int steps = (heads + 4 * hpw - 1) / (4 * hpw);
  int chunks = 1;
  while (chunks < steps && static_cast<long long>(p.T) * chunks < 148 * 8) ++chunks;
  const int chunk_heads = (steps + chunks - 1) / chunks * 4 * hpw;
  chunks = (heads + chunk_heads - 1) / chunk_heads;
  auto kernel = append ? (p.interleaved ? rope_kernel<T, N, true, true> : rope_kernel<T, N, false, true>)
                       : (p.interleaved ? rope_kernel<T, N, true, false> : rope_kernel<T, N, false, false>);
  const long long items = static_cast<long long>(p.T) * chunks;
  return launch_chained(kernel, dim3(static_cast<unsigned>((items + kWarps - 1) / kWarps)), dim3(kThreads), 0, 0, stream,
                        p, chunks, chunk_heads);
}

// The widest vectors (16 bytes at most) that every pointer, stride and section border allows.
template <typename T>
cudaError_t launch_t(const RopeParams& p, cudaStream_t stream) {
  constexpr int kMax = 16 / static_cast<int>(sizeof(T));
  const bool append = p.block_table != nullptr;
  uintptr_t ptrs = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.q_out) |
                   reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.k_out);
  long long el = static_cast<long long>(p.P) | p.q_stride | p.qo_stride | p.k_stride;
  if (append) {
    ptrs |= reinterpret_cast<uintptr_t>(p.v) | reinterpret_cast<uintptr_t>(p.v_out);
    el |= p.v_stride;
  } else {
    el |= p.ko_stride;
  }
  int n = kMax;
  while (n > 1 && (el % n != 0 || p.D % (2 * n) != 0 || ptrs % (n * sizeof(T)) != 0)) n /= 2;
  if (n == 1) return launch_n<T, 1>(p, stream);
  if (n == 2) return launch_n<T, 2>(p, stream);
  if (n == 4) return launch_n<T, 4>(p, stream);
  if constexpr (kMax == 8) return launch_n<T, 8>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace rope

cudaError_t launch_rope(const RopeParams& p, bool f32, cudaStream_t stream) {
  return f32 ? rope::launch_t<float>(p, stream) : rope::launch_t<__nv_bfloat16>(p, stream);
}

}  // namespace da2
