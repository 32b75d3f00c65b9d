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
// Bound by HBM: every element is read and written once, 3 flops each. A CTA takes one token: it
// issues its first loads of q and k (16 bytes per thread and half), computes the token's P angles
// once for all heads while they are in flight, and then turns head after head from shared
// cos/sin. The angle is formed in 64 bits (an integer position times a fp32 frequency needs up to
// 55 bits; at position 1e5 a fp32 product is off by 1e-2 radians), reduced to a fraction of a
// turn there, and only then rounded to fp32 for sincospif.
//
// Append: k goes to the row of its page (token i of sequence b's n_b new ones is logical position
// seqlens[b] - n_b + i) and v beside it, so that neither is written to a buffer in between.

#include "internal.h"
#include "ptx.cuh"

namespace da2 {
namespace rope {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;  // units per thread in flight

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }

// A unit is N pairs of one head (two vectors of N elements), or 2N of its dimensions that pass
// through. Units of a head: P/N rotated ones, then (D - 2P)/(2N) others; a v head has D/(2N)
// others.
template <typename T, int N, bool kInter, bool kAppend>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  extern __shared__ float2 cs[];  // (cos, sin) of the token's P pairs
  __shared__ int s_seq;
  __shared__ long long s_row;
  using V = Vec<T, N>;
  const int t = blockIdx.x;
  const int upr = p.P / N, uph = p.D / (2 * N);  // units per head: rotated, all
  const int units = (p.Hq + p.Hkv * (kAppend ? 2 : 1)) * uph;

  if (kAppend) {
    if (p.cu_seqlens) {
      if (threadIdx.x == 0) s_seq = -1;
      __syncthreads();
      for (int b = threadIdx.x; b < p.B; b += kThreads)
        if (__ldg(p.cu_seqlens + b) <= t && t < __ldg(p.cu_seqlens + b + 1)) s_seq = b;
      __syncthreads();
      if (s_seq < 0) return;  // a row behind the last sequence
    } else if (threadIdx.x == 0) {
      s_seq = t;
    }
    if (threadIdx.x == 0) {
      const int b = s_seq;
      const int end = p.cu_seqlens ? __ldg(p.cu_seqlens + b + 1) : t + 1;
      const int at = __ldg(p.seqlens + b) - (end - t);
      s_row = -1;
      if (at >= 0 && (at >> p.page_shift) < p.max_pages) {
        const int page = __ldg(p.block_table + static_cast<size_t>(b) * p.max_pages + (at >> p.page_shift));
        if (page >= 0 && page < p.num_pages)
          s_row = (static_cast<long long>(page) << p.page_shift) + (at & ((1 << p.page_shift) - 1));
      }
    }
  }

  // where a unit reads and writes; false past the last unit
  auto place = [&](int u, const T*& lo, const T*& hi, T*& wlo, T*& whi, int& c) -> bool {
    if (u >= units) return false;
    const int h = u / uph, r = u - h * uph;
    const T* src;
    T* dst;
    bool rot = r < upr;
    if (h < p.Hq) {
      src = static_cast<const T*>(p.q) + t * p.q_stride + static_cast<size_t>(h) * p.D;
      dst = static_cast<T*>(p.q_out) + t * p.qo_stride + static_cast<size_t>(h) * p.D;
    } else if (!kAppend || h < p.Hq + p.Hkv) {
      const int hk = h - p.Hq;
      src = static_cast<const T*>(p.k) + t * p.k_stride + static_cast<size_t>(hk) * p.D;
      dst = kAppend ? static_cast<T*>(p.k_out) + static_cast<size_t>(hk) * p.D
                    : static_cast<T*>(p.k_out) + t * p.ko_stride + static_cast<size_t>(hk) * p.D;
    } else {
      const int hk = h - p.Hq - p.Hkv;
      src = static_cast<const T*>(p.v) + t * p.v_stride + static_cast<size_t>(hk) * p.D;
      dst = static_cast<T*>(p.v_out) + static_cast<size_t>(hk) * p.D;
      rot = false;
    }
    int a, b;
    if (rot) {
      c = r * N;
      a = kInter ? 2 * c : c;
      b = kInter ? 2 * c + N : p.P + c;
    } else {
      c = -1;
      a = 2 * N * r;  // rotated units cover dimensions 0 .. 2P-1 = 2 N upr
      b = a + N;
    }
    lo = src + a;
    hi = src + b;
    wlo = dst + a;
    whi = dst + b;
    return true;
  };

  bool first = true;
  for (int base = 0; base < units; base += kThreads * kUnroll) {
    V x[kUnroll], y[kUnroll];
    T *wx[kUnroll], *wy[kUnroll];
    int c[kUnroll];
    bool ok[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const T *lo, *hi;
      ok[i] = place(base + i * kThreads + static_cast<int>(threadIdx.x), lo, hi, wx[i], wy[i], c[i]);
      if (ok[i]) {
        x[i] = *reinterpret_cast<const V*>(lo);
        y[i] = *reinterpret_cast<const V*>(hi);
      }
    }
    if (first) {
      for (int j = threadIdx.x; j < p.P; j += kThreads) {
        int axis = 0;
        while (axis + 1 < p.n_axes && j >= p.sec_end[axis]) ++axis;
        double turn = static_cast<double>(__ldg(p.positions + static_cast<size_t>(axis) * p.T + t)) *
                      static_cast<double>(__ldg(p.inv_freq + j)) * 0.15915494309189535;
        turn -= rint(turn);
        float s, co;
        sincospif(static_cast<float>(2.0 * turn), &s, &co);
        cs[j] = make_float2(co, p.inverse ? -s : s);
      }
      __syncthreads();
      first = false;
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (!ok[i]) continue;
      if (c[i] >= 0) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          // element e of the unit's N pairs: (x[e], y[e]), or neighbours when interleaved
          T& a = kInter ? (2 * e < N ? x[i].v[(2 * e) % N] : y[i].v[(2 * e) % N]) : x[i].v[e];
          T& b = kInter ? (2 * e + 1 < N ? x[i].v[(2 * e + 1) % N] : y[i].v[(2 * e + 1) % N]) : y[i].v[e];
          const float2 r = cs[c[i] + e];
          const float fa = to_f32(a), fb = to_f32(b);
          from_f32(fa * r.x - fb * r.y, a);
          from_f32(fb * r.x + fa * r.y, b);
        }
      }
      size_t off = 0;
      if (kAppend) {
        const int h = (base + i * kThreads + static_cast<int>(threadIdx.x)) / uph;
        if (h >= p.Hq) {
          if (s_row < 0) continue;  // no page for this token: only its q is written
          off = static_cast<size_t>(s_row) * p.Hkv * p.D;
        }
      }
      *reinterpret_cast<V*>(wx[i] + off) = x[i];
      *reinterpret_cast<V*>(wy[i] + off) = y[i];
    }
  }
}

template <typename T, int N>
cudaError_t launch_n(const RopeParams& p, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>(p.P) * sizeof(float2);
  const bool append = p.block_table != nullptr;
  auto kernel = append ? (p.interleaved ? rope_kernel<T, N, true, true> : rope_kernel<T, N, false, true>)
                       : (p.interleaved ? rope_kernel<T, N, true, false> : rope_kernel<T, N, false, false>);
  kernel<<<p.T, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
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
