// cache_pages.cu -- the pages of a paged KV cache: take, share, copy, drop and move them.
//
// State, owned by the caller and changed only on the device: block_table [B, max_pages] (page of
// each logical page, -1 none), seqlens [B], refs [num_pages] (how many table entries name a page;
// 0 = free). Serving needs, between the steps of a paged layer: pages for new tokens (extend), a
// second sequence that continues the first (fork: whole pages are shared, a partly filled last
// page is copied so that both can append), the pages that fell between the sinks and the window
// given back (trim), sequences dropped (free), and live pages moved to the front of the pool so
// that its tail can be returned (compact). All of them are a pass over the tables and over refs,
// a few hundred KB: they are bound by the latency of their dependent steps, so each is ONE launch
// of one cluster of eight CTAs that exchange their counts through distributed shared memory and
// need no scratch memory, no second kernel and no host synchronisation.
//
// Free pages are taken lowest index first: the r-th taken page is the r-th free one, found from a
// prefix sum of free counts over warps, CTAs and the cluster, so a result does not depend on
// timing. Counts are changed with atomics, whose integer sums do not depend on their order.
// extend, fork and free are checked before anything is changed and refuse as a whole.

#include <cooperative_groups.h>

#include "bounds.cuh"
#include "internal.h"

namespace da2 {
namespace pages {

namespace cg = cooperative_groups;

constexpr int kCtas = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kAllWarps = kCtas * kWarps;
constexpr int kAllThreads = kCtas * kThreads;

struct Shared {
  int cnt[kWarps];      // of each warp of this CTA
  int flag;             // this CTA found a reason to refuse
  int scan[kWarps];
  int2 in[2][kCtas];    // what each CTA of the cluster sent: (sum, flag), by exchange
};

// Pages [lo, hi) of warp `w` of the cluster: consecutive, a multiple of 32 long.
__device__ __forceinline__ void warp_range(int num_pages, int w, int& lo, int& hi) {
  const int per = ((num_pages + kAllWarps - 1) / kAllWarps + 31) / 32 * 32;
  lo = static_cast<int>(min(static_cast<long long>(w) * per, static_cast<long long>(num_pages)));
  hi = static_cast<int>(min(static_cast<long long>(lo) + per, static_cast<long long>(num_pages)));
}

// Number of pages p of [lo, hi) with (refs[p] > 0) == live; all lanes get it.
__device__ __forceinline__ int count_pages(const int32_t* refs, int lo, int hi, bool live, int lane) {
  int n = 0;
#pragma unroll 8
  for (int p = lo + lane; p < hi; p += 32) n += (refs[p] > 0) == live ? 1 : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// One value per warp and one flag per CTA, for all of the cluster: returns the sum of the warps before
// this one, the total and whether any flag is set. Every CTA stores its sum and flag into the shared
// memory of all eight, so that one barrier is enough: nothing is read from another CTA after it, and no
// CTA needs to wait for others before it exits. (Leaving them to be read took a barrier before and one
// after, and a trip between SMs in between.) The barrier also orders all that any CTA read before it
// ahead of all that is written after it. `slot`: 0 or 1, another for each exchange of a kernel. The
// first exchange follows cluster_arrive_relaxed at the kernel's start.
__device__ __forceinline__ int exchange(Shared& sh, int slot, int mine, int& total, bool& flag) {
  cg::cluster_group cl = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sh.cnt[warp] = mine;
  __syncthreads();
  int base = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += sh.cnt[w];
    sum += sh.cnt[w];
  }
  const int rank = static_cast<int>(cl.block_rank());
  if (slot == 0) cluster_wait();  // every CTA is running
  if (threadIdx.x < kCtas) *cl.map_shared_rank(&sh.in[slot][rank], threadIdx.x) = make_int2(sum, sh.flag);
  cl.sync();
  total = 0;
  flag = false;
#pragma unroll
  for (int r = 0; r < kCtas; ++r) {
    const int2 v = sh.in[slot][r];
    if (r < rank) base += v.x;
    total += v.x;
    flag |= v.y != 0;
  }
  return base;
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// In-place inclusive prefix sum of a[0..n) in shared memory by the CTA.
__device__ __forceinline__ void block_scan(Shared& sh, int* a, int n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int carry = 0;
  for (int b = 0; b < n; b += kThreads) {
    const int i = b + threadIdx.x;
    int v = i < n ? a[i] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) sh.scan[warp] = v;
    __syncthreads();
    int before = carry, sum = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.scan[w];
      sum += sh.scan[w];
    }
    if (i < n) a[i] = v + before;
    carry += sum;
    __syncthreads();
  }
}

// First index of the inclusive prefix sums pre[0..n) whose sum exceeds r.
__device__ __forceinline__ int owner_of(const int* pre, int n, int r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] > r) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Calls take(rank, page) for the free pages of this warp's range whose rank is below `want`.
template <typename F>
__device__ __forceinline__ void take_free(const int32_t* refs, int lo, int hi, int base, int want, int lane, F take) {
  for (int p0 = lo; p0 < hi && base < want; p0 += 32) {
    const int p = p0 + lane;
    const bool free = p < hi && refs[p] <= 0;
    const unsigned m = __ballot_sync(0xffffffffu, free);
    const int rank = base + __popc(m & ((1u << lane) - 1u));
    if (free && rank < want) take(rank, p);
    base += __popc(m);
  }
}

// One table entry fewer names page e: 1 if it became free. A count that was 0 already stays 0.
__device__ __forceinline__ int release(int32_t* refs, int num_pages, int e) {
  if (e < 0 || e >= num_pages) return 0;
  const int old = atomicSub(refs + e, 1);
  if (old <= 0) atomicAdd(refs + e, 1);
  return old == 1 ? 1 : 0;
}

__device__ __forceinline__ int pages_of(int len, int shift) { return (max(len, 0) + (1 << shift) - 1) >> shift; }

// ---------------------------------------------------------------------------------- extend
__global__ void __launch_bounds__(kThreads)
extend_kernel(int32_t* table, int32_t* seqlens, int32_t* refs, const int32_t* n_new, int32_t* result, int B,
              int max_pages, int shift, int num_pages, int* err) {
  pdl_wait();
  cluster_arrive_relaxed();
  __shared__ Shared sh;
  __shared__ int pre[kMaxCacheSeqs], first[kMaxCacheSeqs];
  if (!checked(B > 0 && B <= kMaxCacheSeqs, err)) return;  // (the whole cluster)
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31, gw = static_cast<int>(cl.block_rank()) * kWarps + (threadIdx.x >> 5);
  if (threadIdx.x == 0) sh.flag = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += kThreads) {
    const int old = max(seqlens[b], 0), add = max(n_new[b], 0);
    const long long end = static_cast<long long>(old) + add;
    if (end > (static_cast<long long>(max_pages) << shift)) {
      sh.flag = 1;  // more tokens than the row has pages for
      pre[b] = 0;
    } else {
      pre[b] = pages_of(static_cast<int>(end), shift) - pages_of(old, shift);
    }
    first[b] = pages_of(old, shift);
  }
  __syncthreads();
  block_scan(sh, pre, B);
  const int want = pre[B - 1];
  int lo, hi, total;
  bool bad;
  warp_range(num_pages, gw, lo, hi);
  const int base = exchange(sh, 0, count_pages(refs, lo, hi, false, lane), total, bad);
  const bool refuse = bad || want > total;
  if (!refuse) {
    take_free(refs, lo, hi, base, want, lane, [&](int r, int p) {
      const int b = owner_of(pre, B, r);
      const int at = first[b] + r - (b > 0 ? pre[b - 1] : 0);
      if (!checked(at >= 0 && at < max_pages && p < num_pages, err)) return;
      table[static_cast<size_t>(b) * max_pages + at] = p;
      refs[p] = 1;
    });
    if (cl.block_rank() == 0)
      for (int b = threadIdx.x; b < B; b += kThreads) seqlens[b] = max(seqlens[b], 0) + max(n_new[b], 0);
  }
  if (cl.block_rank() == 0 && threadIdx.x == 0) result[0] = refuse ? -1 : want;
}

// ------------------------------------------------------------------------------------ fork
__global__ void __launch_bounds__(kThreads)
fork_kernel(int32_t* table, int32_t* seqlens, int32_t* refs, const int32_t* parents, const int32_t* children,
            int2* copies, int32_t* result, int n, int B, int max_pages, int shift, int num_pages, int* err) {
  pdl_wait();
  cluster_arrive_relaxed();
  __shared__ Shared sh;
  __shared__ int pre[kMaxCacheSeqs], kid[kMaxCacheSeqs], len[kMaxCacheSeqs];
  if (!checked(n > 0 && n <= kMaxCacheSeqs, err)) return;  // (the whole cluster)
  cg::cluster_group cl = cg::this_cluster();
  const int rank = static_cast<int>(cl.block_rank());
  const int lane = threadIdx.x & 31, gw = rank * kWarps + (threadIdx.x >> 5);
  const int gt = rank * kThreads + threadIdx.x;
  if (threadIdx.x == 0) sh.flag = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int a = parents[i], c = children[i];
    kid[i] = -1;  // padding
    len[i] = 0;
    if (a >= 0 && c >= 0) {
      if (a >= B || c >= B || a == c || seqlens[c] != 0 || seqlens[a] < 0 || pages_of(seqlens[a], shift) > max_pages) {
        sh.flag = 1;
      } else {
        kid[i] = c;
        len[i] = seqlens[a];
      }
    }
    pre[i] = (len[i] & ((1 << shift) - 1)) != 0 ? 1 : 0;
  }
  __syncthreads();
  // the same child twice
  for (int i = gt; i < n; i += kAllThreads)
    if (kid[i] >= 0)
      for (int j = 0; j < i; ++j)
        if (kid[j] == kid[i]) sh.flag = 1;
  block_scan(sh, pre, n);
  const int want = pre[n - 1];
  int lo, hi, total;
  bool bad;
  warp_range(num_pages, gw, lo, hi);
  const int base = exchange(sh, 0, count_pages(refs, lo, hi, false, lane), total, bad);
  const bool refuse = bad || want > total;
  if (!refuse) {
    // a page of its own for each partly filled last page
    take_free(refs, lo, hi, base, want, lane, [&](int r, int p) {
      const int i = owner_of(pre, n, r);
      const int at = len[i] >> shift;
      if (!checked(i < n && at < max_pages && p < num_pages && parents[i] < B && kid[i] >= 0 && kid[i] < B, err)) return;
      const int src = table[static_cast<size_t>(parents[i]) * max_pages + at];
      copies[i] = src >= 0 && src < num_pages ? make_int2(src, p) : make_int2(-1, -1);
      table[static_cast<size_t>(kid[i]) * max_pages + at] = p;
      refs[p] = 1;
    });
    // the whole pages are shared: items of 128 entries of one pair
    const int per = (max_pages + 127) / 128;
    for (long long it = gw; it < static_cast<long long>(n) * per; it += kAllWarps) {
      const int i = static_cast<int>(it / per), l0 = static_cast<int>(it % per) * 128;
      const int whole = len[i] >> shift;
      if (kid[i] < 0) continue;
      const int32_t* from = table + static_cast<size_t>(parents[i]) * max_pages;
      int32_t* to = table + static_cast<size_t>(kid[i]) * max_pages;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int l = l0 + 32 * u + lane;
        if (l < whole && checked(l < max_pages, err)) {
          const int e = from[l];
          to[l] = e;
          if (e >= 0 && e < num_pages) atomicAdd(refs + e, 1);
        }
      }
    }
    if (rank == 0)
      for (int i = threadIdx.x; i < n; i += kThreads)
        if (kid[i] >= 0) seqlens[kid[i]] = len[i];
  }
  for (int i = gt; i < n; i += kAllThreads)
    if (refuse || pre[i] == (i > 0 ? pre[i - 1] : 0)) copies[i] = make_int2(-1, -1);
  if (gt == 0) result[0] = bad ? -2 : (refuse ? -1 : want);
}

// ------------------------------------------------------------------------------------ trim
__global__ void __launch_bounds__(kThreads)
trim_kernel(int32_t* table, const int32_t* seqlens, int32_t* refs, int32_t* result, int B, int max_pages, int shift,
            int num_pages, int window, int keep, int* err) {
  pdl_wait();
  cluster_arrive_relaxed();
  __shared__ Shared sh;
  if (threadIdx.x == 0) sh.flag = 0;
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  const int gw = static_cast<int>(cl.block_rank()) * kWarps + (threadIdx.x >> 5);
  // items of 128 entries of one sequence's row
  const int per = (max_pages + 127) / 128;
  int freed = 0;
  for (long long it = gw; it < static_cast<long long>(B) * per; it += kAllWarps) {
    const int b = static_cast<int>(it / per), l0 = static_cast<int>(it % per) * 128;
    const int end = min(max(max(seqlens[b], 0) - window, 0) >> shift, max_pages);
    if (l0 >= end || l0 + 128 <= keep) continue;
    int32_t* row = table + static_cast<size_t>(b) * max_pages;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int l = l0 + 32 * u + lane;
      if (l >= keep && l < end && checked(b < B && l >= 0 && l < max_pages, err)) {
        const int e = row[l];
        if (e >= 0) {
          row[l] = -1;
          freed += release(refs, num_pages, e);
        }
      }
    }
  }
  int total;
  bool none;
  exchange(sh, 0, warp_sum(freed), total, none);
  if (cl.block_rank() == 0 && threadIdx.x == 0) result[0] = total;
}

// ------------------------------------------------------------------------------------ free
__global__ void __launch_bounds__(kThreads)
free_kernel(int32_t* table, int32_t* seqlens, int32_t* refs, const int32_t* seqs, int32_t* result, int n, int B,
            int max_pages, int num_pages, int* err) {
  pdl_wait();
  cluster_arrive_relaxed();
  __shared__ Shared sh;
  if (threadIdx.x == 0) sh.flag = 0;
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cl.block_rank());
  const int gw = rank * kWarps + (threadIdx.x >> 5), gt = rank * kThreads + threadIdx.x;
  // every CTA looks at the whole list, so that none has to ask another before it changes anything
  int found = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) found |= seqs[i] >= B ? 1 : 0;
  const bool bad = __syncthreads_or(found) != 0;
  int freed = 0;
  if (!bad) {
    const int per = (max_pages + 127) / 128;
    for (long long it = gw; it < static_cast<long long>(n) * per; it += kAllWarps) {
      const int b = seqs[it / per], l0 = static_cast<int>(it % per) * 128;
      if (b < 0) continue;  // padding
      if (!checked(b < B, err)) continue;
      int32_t* row = table + static_cast<size_t>(b) * max_pages;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int l = l0 + 32 * u + lane;
        // exchanged, so that a sequence listed twice gives its pages back once
        if (l < max_pages && row[l] >= 0) freed += release(refs, num_pages, atomicExch(row + l, -1));
      }
      if (l0 == 0 && lane == 0) seqlens[b] = 0;
    }
  }
  int total;
  bool none;
  exchange(sh, 0, warp_sum(freed), total, none);
  if (gt == 0) result[0] = bad ? -2 : total;
}

// --------------------------------------------------------------------------------- compact
// n live pages; the r-th live page at or behind n goes to the r-th free one before it.
__global__ void __launch_bounds__(kThreads)
compact_kernel(const int32_t* table, const int32_t* refs, int32_t* table_out, int32_t* refs_out, int2* moves,
               int32_t* result, int B, int max_pages, int num_pages, int* err) {
  pdl_wait();
  cluster_arrive_relaxed();
  __shared__ Shared sh;
  if (threadIdx.x == 0) sh.flag = 0;
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cl.block_rank());
  const int gw = rank * kWarps + (threadIdx.x >> 5), gt = rank * kThreads + threadIdx.x;
  int lo, hi, n;
  bool none;
  warp_range(num_pages, gw, lo, hi);
  const int base = exchange(sh, 0, count_pages(refs, lo, hi, true, lane), n, none);
  // live pages before n: those of this warp's range, summed over the cluster
  int before = 0;
  exchange(sh, 1, lo < n ? count_pages(refs, lo, min(hi, n), true, lane) : 0, before, none);
  const int n_moves = n - before;
  int2* mv = moves;
  int r_live = base;
  for (int p0 = lo; p0 < hi; p0 += 32) {
    const int p = p0 + lane;
    const bool live = p < hi && refs[p] > 0;
    const unsigned m = __ballot_sync(0xffffffffu, live);
    const int lr = r_live + __popc(m & ((1u << lane) - 1u));  // live pages before p
    if (p < hi) {
      const int at = live ? lr - before : p - lr;
      if (live != (p < n) && checked(at >= 0 && at < num_pages / 2, err)) (live ? mv[at].x : mv[at].y) = p;
    }
    r_live += __popc(m);
  }
  for (int r = n_moves + gt; r < num_pages / 2; r += kAllThreads) mv[r] = make_int2(-1, -1);
  __threadfence();
  cl.sync();  // the moves are complete, and every CTA has read refs
  for (int p = gt; p < num_pages; p += kAllThreads) {
    // pages that stay: live ones before n; free ones behind it stay free
    const int c = refs[p];
    if (p < n ? c > 0 : c <= 0) refs_out[p] = p < n ? c : 0;
  }
  for (int r = gt; r < n_moves; r += kAllThreads) {
    const int2 m = __ldcg(mv + r);
    if (!checked(m.x >= 0 && m.x < num_pages && m.y >= 0 && m.y < num_pages, err)) continue;
    const int c = refs[m.x];
    refs_out[m.y] = c;
    refs_out[m.x] = 0;
  }
  for (long long i = gt; i < static_cast<long long>(B) * max_pages; i += kAllThreads) {
    int e = table[i];
    if (e >= n && n_moves > 0) {
      // its move: the sources ascend
      int a = 0, b = n_moves - 1;
      while (a < b) {
        const int mid = (a + b) >> 1;
        if (__ldcg(&mv[mid].x) < e) a = mid + 1; else b = mid;
      }
      const int2 m = __ldcg(mv + a);
      if (m.x == e) e = m.y;
    }
    table_out[i] = e;
  }
  if (gt == 0) result[0] = n;
}

// ------------------------------------------------------------------------------ copy pages
// One page each of the K and the V cache per listed (source, destination); entries out of range
// are skipped. Bound by HBM: 16 KB pieces, four 16-byte loads per thread in flight, the CTAs walk
// the list together so that a list of a few pages still uses the whole GPU.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kPieceVecs = kCopyThreads * kCopyUnroll;

__global__ void __launch_bounds__(kCopyThreads)
copy_kernel(uint4* k, uint4* v, const int2* copies, int n, int num_pages,
            int page_vecs, int pieces, int* err) {
  pdl_wait();
  const long long items = static_cast<long long>(n) * 2 * pieces;
  long long it = blockIdx.x;
  if (it >= items) return;
  int2 next = *(copies + it / pieces / 2);
  for (; it < items; it += gridDim.x) {
    const int2 c = next;
    if (it + gridDim.x < items) next = *(copies + (it + gridDim.x) / pieces / 2);  // while this piece is copied
    if (c.x < 0 || c.y < 0 || c.x >= num_pages || c.y >= num_pages) continue;
    uint4* pool = (it / pieces) & 1 ? v : k;
    const uint4* src = pool + static_cast<size_t>(c.x) * page_vecs;
    uint4* dst = pool + static_cast<size_t>(c.y) * page_vecs;
    const int at = static_cast<int>(it % pieces) * kPieceVecs + threadIdx.x;
    if (!checked(it / pieces / 2 < n && at >= 0, err)) continue;
    uint4 x[kCopyUnroll];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (at + i * kCopyThreads < page_vecs) x[i] = __ldcs(src + at + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
      if (at + i * kCopyThreads < page_vecs) __stcs(dst + at + i * kCopyThreads, x[i]);
  }
}

}  // namespace pages

cudaError_t launch_cache_extend(int32_t* table, int32_t* seqlens, int32_t* refs, const int32_t* n_new,
                                int32_t* result, int B, int max_pages, int page_shift, int num_pages,
                                cudaStream_t stream) {
  int* err = nullptr;
  if (const cudaError_t e = bounds_error_word(&err); e != cudaSuccess) return e;
  return launch_chained(pages::extend_kernel, dim3(pages::kCtas), dim3(pages::kThreads), 0, pages::kCtas, stream,
                        table, seqlens, refs, n_new, result, B, max_pages, page_shift, num_pages, err);
}

cudaError_t launch_cache_fork(int32_t* table, int32_t* seqlens, int32_t* refs, const int32_t* parents,
                              const int32_t* children, int32_t* copies, int32_t* result, int n, int B, int max_pages,
                              int page_shift, int num_pages, cudaStream_t stream) {
  int* err = nullptr;
  if (const cudaError_t e = bounds_error_word(&err); e != cudaSuccess) return e;
  return launch_chained(pages::fork_kernel, dim3(pages::kCtas), dim3(pages::kThreads), 0, pages::kCtas, stream,
                        table, seqlens, refs, parents, children, reinterpret_cast<int2*>(copies), result, n, B,
                        max_pages, page_shift, num_pages, err);
}

cudaError_t launch_cache_trim(int32_t* table, const int32_t* seqlens, int32_t* refs, int32_t* result, int B,
                              int max_pages, int page_shift, int num_pages, int window, int sink,
                              cudaStream_t stream) {
  int* err = nullptr;
  if (const cudaError_t e = bounds_error_word(&err); e != cudaSuccess) return e;
  const int keep = static_cast<int>((static_cast<long long>(sink) + (1 << page_shift) - 1) >> page_shift);
  return launch_chained(pages::trim_kernel, dim3(pages::kCtas), dim3(pages::kThreads), 0, pages::kCtas, stream,
                        table, seqlens, refs, result, B, max_pages, page_shift, num_pages, window, keep, err);
}

cudaError_t launch_cache_free(int32_t* table, int32_t* seqlens, int32_t* refs, const int32_t* seqs, int32_t* result,
                              int n, int B, int max_pages, int num_pages, cudaStream_t stream) {
  int* err = nullptr;
  if (const cudaError_t e = bounds_error_word(&err); e != cudaSuccess) return e;
  return launch_chained(pages::free_kernel, dim3(pages::kCtas), dim3(pages::kThreads), 0, pages::kCtas, stream,
                        table, seqlens, refs, seqs, result, n, B, max_pages, num_pages, err);
}

cudaError_t launch_cache_compact(const int32_t* table, const int32_t* refs, int32_t* table_out, int32_t* refs_out,
                                 int32_t* moves, int32_t* result, int B, int max_pages, int num_pages,
                                 cudaStream_t stream) {
  int* err = nullptr;
  if (const cudaError_t e = bounds_error_word(&err); e != cudaSuccess) return e;
  return launch_chained(pages::compact_kernel, dim3(pages::kCtas), dim3(pages::kThreads), 0, pages::kCtas, stream,
                        table, refs, table_out, refs_out, reinterpret_cast<int2*>(moves), result, B, max_pages,
                        num_pages, err);
}

cudaError_t launch_cache_copy_pages(void* k, void* v, const int32_t* copies, int n, int num_pages, size_t page_bytes,
                                    cudaStream_t stream) {
  const int page_vecs = static_cast<int>(page_bytes / 16);
  const int pieces = (page_vecs + pages::kPieceVecs - 1) / pages::kPieceVecs;
  int device = 0, n_sms = 0;
  int* err = nullptr;
  cudaError_t e = bounds_error_word(&err);
  if (e != cudaSuccess) return e;
  e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&n_sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return e;
  const long long items = static_cast<long long>(n) * 2 * pieces;
  // Many short-lived CTAs: 994 pages of 128 KB in both caches took 80 us (521 MB, 6.5 TB/s) with 64 CTAs
  // for every SM, 95 with the 8 that are resident at a time.
  const long long most = 64LL * n_sms;
  return launch_chained(pages::copy_kernel, dim3(static_cast<unsigned>(items < most ? items : most)),
                        dim3(pages::kCopyThreads), 0, 0, stream, static_cast<uint4*>(k), static_cast<uint4*>(v),
                        reinterpret_cast<const int2*>(copies), n, num_pages, page_vecs, pieces, err);
}

}  // namespace da2
