// Stable counting sort by a digit of up to 1024 bins, the step that the plan
// of an expert exchange (one digit: the expert) and the embedding's gradient
// (two or three digits of the token) share.
//
// A CTA of 32 warps takes a chunk of items; a warp takes a run of the chunk's
// items in order, 32 at a time, so an item's place among its equals is: equals
// in earlier chunks + in earlier warps + in earlier steps of its warp + in
// lower lanes.  Lanes with equal digits find each other with one match; only
// the lowest of them touches the warp's counter, so no atomics order anything.
#pragma once

#include "ops_common.cuh"

namespace pl {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortIpt = 8;          // items per thread, at most
constexpr int kSortBins = 1024;      // bins of one digit, at most; one more for dropped items
constexpr uint64_t kSortSmall = 8192;  // items that one CTA sorts by itself

// Items of one CTA's chunk: 1024 for every started 152 x 1024, so that the
// chunks fill the SMs once, up to 8192; more items take more chunks.
inline uint64_t sort_chunk(uint64_t n) {
  const uint64_t per = (n + 152 * kSortThreads - 1) / (152 * kSortThreads);
  return (uint64_t)kSortThreads * std::max<uint64_t>(1, std::min<uint64_t>(per, kSortIpt));
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
  for (int b = threadIdx.x; b < bins; b += blockDim.x) {
    uint32_t sum = 0;
    for (int w = 0; w < warps; ++w) {
      const uint32_t c = cnt[w * bins + b];
      cnt[w * bins + b] = (uint16_t)sum;
      sum += c;
    }
    each(b, sum);
  }
  __syncthreads();
}

// Sums of the chunks' counts (rows of `bins` words, one per chunk): all[b] over
// every chunk, before[b] over the chunks before this one.
__device__ __forceinline__ void sum_chunks(const uint32_t* counts, uint32_t chunks, uint32_t chunk, int bins, uint32_t* all,
                                           uint32_t* before) {
  for (int b = threadIdx.x; b < bins; b += blockDim.x) all[b] = before[b] = 0;
  __syncthreads();
  const int parts = max(1, (int)blockDim.x / bins);
  const int part = threadIdx.x / bins;
  for (int b = threadIdx.x - part * bins; part < parts && b < bins; b += blockDim.x) {
    uint32_t s = 0, sb = 0;
#pragma unroll 8
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

}  // namespace pl
