// Stable counting sort by a digit of up to 1024 bins, the step that the plan
// of an expert exchange (one digit: the expert) and the embedding's gradient
// (two or three digits of the token) share.
//
// A CTA takes a chunk of items; a warp takes a run of the chunk's items in
// order, 32 at a time, so an item's place among its equals is: equals in earlier
// chunks + in earlier warps + in earlier steps of its warp + in lower lanes.
// Lanes with equal digits find each other with one match; only the lowest of
// them touches the warp's counter, so no atomics order anything.  (The kernel
// that counts lets the one that places start at once; that one does what needs
// no counts and then waits for them.  What it reads before is older than the
// counting kernel, which lets it start only after its own op_wait.)
#pragma once

#include <cooperative_groups.h>

#include "ops_common.cuh"

namespace pl {

constexpr int kSortThreads = 512;    // of a chunk's CTA
constexpr int kSortIpt = 8;          // items per thread, at most
constexpr int kSortBins = 1024;      // bins of one digit, at most; one more for dropped items

// Up to kClusterSort items are sorted by one cluster in one launch: its CTAs
// keep the items in shared memory and read each other's counts there.  More go
// through two launches a digit, one that counts and one that places.  (A plan
// with 65 bins: 8192 items 6.0 us by one cluster and 7.0 in two launches, 16384
// items 6.3 and 7.5, 32768 items 8.3 and 8.1; with 257 bins, 65536 items 18 and 11.)
constexpr int kClusterThreads = 1024;
constexpr int kClusterMost = 8;
constexpr uint64_t kClusterSort = (uint64_t)kClusterThreads * kClusterMost * 2;

// CTAs of the cluster and items per thread (powers of two) for n items: a CTA
// for every started 1024 x each, then more items per thread.
struct ClusterShape {
  int ctas = 1, ipt = 1;
  explicit ClusterShape(uint64_t n, int each = 2) {
    while (ctas < kClusterMost && n > (uint64_t)ctas * each * kClusterThreads) ctas *= 2;
    while (n > (uint64_t)ctas * ipt * kClusterThreads) ipt *= 2;
  }
};

// Items of one CTA's chunk: 1024, or more where 152 x 1024 do not hold them,
// so that the chunks fill the SMs once, up to 4096; then there are more chunks.
inline uint64_t sort_chunk(uint64_t n) {
  const uint64_t per = (n + 152 * kSortThreads - 1) / (152 * kSortThreads);
  return (uint64_t)kSortThreads * std::max<uint64_t>(2, std::min<uint64_t>(per, kSortIpt));
}
inline uint64_t sort_chunks(uint64_t n) { return (n + sort_chunk(n) - 1) / sort_chunk(n); }

// Exclusive sums over `bins` (at most blockDim.x) values, one per thread; every
// thread calls it.  `tmp`: 33 words of shared memory.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* tmp, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  uint32_t s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
    if (lane >= d) s += o;
  }
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = lane < warps ? tmp[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, w, d);
      if (lane >= d) w += o;
    }
    tmp[lane] = w;
  }
  __syncthreads();
  const uint32_t before = warp ? tmp[warp - 1] : 0;
  *total = tmp[warps - 1];
  __syncthreads();
  return before + s - v;
}

// Local places of a chunk's items.  digit[q] is the thread's item q's bin
// (< bins), item (warp * ipt + q) * 32 + lane of the chunk, or -1 past the
// end.  Afterwards local[q] counts the item's equals earlier in its warp and
// cnt[w * bins + b] the items of bin b in warps before w; `each(b, n)` is
// called once for every bin with the chunk's count.
template <typename F>
__device__ __forceinline__ void rank_chunk(const int (&digit)[kSortIpt], uint32_t (&local)[kSortIpt], int ipt, int bins,
                                           uint16_t* cnt, F each) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int i = threadIdx.x; i < warps * bins; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  uint16_t* mine = cnt + warp * bins;
#pragma unroll
  for (int q = 0; q < kSortIpt; ++q) {
    if (q < ipt) {
      const unsigned peers = __match_any_sync(0xFFFFFFFFu, digit[q]);
      const int lower = __popc(peers & ((1u << lane) - 1u));
      uint32_t before = 0;
      if (digit[q] >= 0) before = mine[digit[q]];
      __syncwarp();
      if (digit[q] >= 0 && lower == 0) mine[digit[q]] = (uint16_t)(before + __popc(peers));
      __syncwarp();
      local[q] = before + lower;
    }
  }
  __syncthreads();
  // eight counts of a bin are loaded before their sums are stored: one by one,
  // each load would wait for the sum before it
  for (int b = threadIdx.x; b < bins; b += blockDim.x) {
    uint32_t sum = 0;
    for (int w0 = 0; w0 < warps; w0 += 8) {
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = w0 + i < warps ? cnt[(w0 + i) * bins + b] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (w0 + i < warps) cnt[(w0 + i) * bins + b] = (uint16_t)sum;
        sum += c[i];
      }
    }
    each(b, sum);
  }
  __syncthreads();
}

// Sums of the chunks' counts (rows of `bins` words, one per chunk): all[b] over
// every chunk, before[b] over the chunks before this one.
__device__ __forceinline__ void sum_chunks(const uint32_t* counts, uint32_t chunks, uint32_t chunk, int bins,
                                           uint32_t* all, uint32_t* before) {
  for (int b = threadIdx.x; b < bins; b += blockDim.x) all[b] = before[b] = 0;
  __syncthreads();
  const int parts = max(1, (int)blockDim.x / bins);
  const int part = threadIdx.x / bins;
  for (int b = threadIdx.x - part * bins; part < parts && b < bins; b += blockDim.x) {
    uint32_t s = 0, sb = 0;
#pragma unroll 16
    for (uint32_t c = part; c < chunks; c += parts) {
      const uint32_t v = __ldcg(counts + (uint64_t)c * bins + b);
      s += v;
      if (c < chunk) sb += v;
    }
    atomicAdd(all + b, s);  // whole numbers: the order does not matter
    atomicAdd(before + b, sb);
  }
  __syncthreads();
}

// base[b] = the first place of this CTA's items of bin b: items of lower bins in
// the whole cluster, and those of bin b in the CTAs before.  `hist`: this CTA's
// counts, at the same place in every CTA of the cluster.  total: all items.
__device__ __forceinline__ uint32_t cluster_bases(uint32_t* hist, int bins, uint32_t* base, uint32_t* tmp) {
  const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int ctas = (int)cluster.num_blocks(), me = (int)cluster.block_rank();
  cluster.sync();
  uint32_t carry = 0;
  for (int b0 = 0; b0 < bins; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    uint32_t all = 0, before = 0;
    if (b < bins) {
      uint32_t v[kClusterMost];
#pragma unroll
      for (int r = 0; r < kClusterMost; ++r) v[r] = r < ctas ? cluster.map_shared_rank(hist, r)[b] : 0;
#pragma unroll
      for (int r = 0; r < kClusterMost; ++r) {
        all += v[r];
        before += r < me ? v[r] : 0;
      }
    }
    uint32_t total;
    const uint32_t at = carry + block_exclusive(all, tmp, &total);
    if (b < bins) base[b] = at + before;
    carry += total;
  }
  __syncthreads();
  return carry;
}

}  // namespace pl
