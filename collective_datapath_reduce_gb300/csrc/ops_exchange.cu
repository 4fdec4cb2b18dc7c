// The exchange of token rows with experts: the plan (a stable sort of the
// picks by expert), the copy of rows by it, the weighted sum back, and the
// sum's gradient.  The copies are a copy Atom whose destinations are named by
// index, the sum an N-to-1 reduce Atom whose sources are.
#include <type_traits>

#include "kernels_bulk.cuh"
#include "ops_common.cuh"
#include "ops_sort.cuh"

namespace pl {
namespace {

// ------------------------------------------------------------------- plan

__device__ __forceinline__ int expert_of(const int32_t* ids, uint64_t i, uint64_t n, int experts) {
  if (i >= n) return -1;
  const int e = ids[i];
  return e >= 0 && e < experts ? e : experts;  // bin `experts`: dropped
}

// Counts of a chunk's picks by expert; dropped ones are not counted.
__global__ void __launch_bounds__(kSortThreads) plan_count_kernel(const __grid_constant__ PlanArgs a, uint32_t chunk) {
  op_wait();
  op_next();
  __shared__ uint32_t hist[kSortBins + 1];
  for (int b = threadIdx.x; b <= a.experts; b += blockDim.x) hist[b] = 0;
  __syncthreads();
  const uint64_t i0 = (uint64_t)blockIdx.x * chunk;
  for (uint32_t i = threadIdx.x; i < chunk; i += blockDim.x) {
    const int e = expert_of(a.ids, i0 + i, a.slots, a.experts);
    if (e >= 0) atomicAdd(hist + e, 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < a.experts; b += blockDim.x) a.counts[(uint64_t)blockIdx.x * a.experts + b] = hist[b];
}

__device__ __forceinline__ void store_places(const PlanArgs& a, uint64_t i0, int ipt, const int (&digit)[kSortIpt],
                                             const uint32_t (&local)[kSortIpt], const uint32_t* base, const uint16_t* cnt) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int q = 0; q < kSortIpt; ++q) {
    if (q < ipt && digit[q] >= 0) {
      const uint64_t i = i0 + (uint64_t)(warp * ipt + q) * 32 + lane;
      const int32_t p = (int32_t)(base[digit[q]] + cnt[warp * (a.experts + 1) + digit[q]] + local[q]);
      a.places[i] = digit[q] == a.experts ? ~p : p;
    }
  }
}

// One chunk's places, of many.
__global__ void __launch_bounds__(kSortThreads) plan_place_kernel(const __grid_constant__ PlanArgs a, uint32_t chunk, int ipt) {
  extern __shared__ uint16_t cnt[];
  __shared__ uint32_t base[kSortBins + 1], before[kSortBins], tmp[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t i0 = (uint64_t)blockIdx.x * chunk;
  int digit[kSortIpt];
  uint32_t local[kSortIpt];
#pragma unroll
  for (int q = 0; q < kSortIpt; ++q)
    if (q < ipt) digit[q] = expert_of(a.ids, i0 + (uint64_t)(warp * ipt + q) * 32 + lane, a.slots, a.experts);
  rank_chunk(digit, local, ipt, a.experts + 1, cnt, [](int, uint32_t) {});
  op_wait();
  op_next();
  sum_chunks(a.counts, gridDim.x, blockIdx.x, a.experts, base, before);
  uint32_t carry = 0, earlier = 0;  // picks with an expert: all, and those of earlier chunks
  for (int b0 = 0; b0 < a.experts; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const uint32_t n = b < a.experts ? base[b] : 0, m = b < a.experts ? before[b] : 0;
    uint32_t total, more;
    const uint32_t at = carry + block_exclusive(n, tmp, &total);
    block_exclusive(m, tmp, &more);
    if (b < a.experts) {
      base[b] = at + m;
      if (blockIdx.x == 0) a.offsets[b] = (int32_t)at;
    }
    carry += total;
    earlier += more;
  }
  if (threadIdx.x == 0) {
    base[a.experts] = carry + (uint32_t)(i0 - earlier);  // dropped picks follow all others
    if (blockIdx.x == 0) a.offsets[a.experts] = (int32_t)carry;
  }
  __syncthreads();
  store_places(a, i0, ipt, digit, local, base, cnt);
}

// All places, by one cluster.
__global__ void __launch_bounds__(kClusterThreads) plan_cluster_kernel(const __grid_constant__ PlanArgs a, int ipt) {
  op_wait();
  op_next();
  extern __shared__ uint16_t cnt[];
  __shared__ uint32_t hist[kSortBins + 1], base[kSortBins + 1], tmp[33];
  const int bins = a.experts + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t i0 = (uint64_t)blockIdx.x * blockDim.x * ipt;
  int digit[kSortIpt];
  uint32_t local[kSortIpt];
#pragma unroll
  for (int q = 0; q < kSortIpt; ++q)
    if (q < ipt) digit[q] = expert_of(a.ids, i0 + (uint64_t)(warp * ipt + q) * 32 + lane, a.slots, a.experts);
  rank_chunk(digit, local, ipt, bins, cnt, [&](int b, uint32_t n) { hist[b] = n; });
  cluster_bases(hist, bins, base, tmp);
  if (blockIdx.x == 0)  // the first CTA has no items before it: its bases are the experts'
    for (int b = threadIdx.x; b < bins; b += blockDim.x) a.offsets[b] = (int32_t)base[b];
  store_places(a, i0, ipt, digit, local, base, cnt);
  cooperative_groups::this_cluster().sync();  // the counts stay until all have read them
}

// ------------------------------------------------------------ rows by index

// A CTA holds `per` groups of tpt threads (a multiple of 32); each group takes
// U tokens and keeps one vector of each in flight.  The picks of the CTA's
// tokens are read once, into shared memory.
constexpr int kMostTokens = 8 * 4;
struct Picks {
  int64_t row[kMostTokens * PURLIN_MAX_TOP_K];  // the row, ~row of a dropped pick, kNoRow outside
  float w[kMostTokens * PURLIN_MAX_TOP_K];
};
constexpr int64_t kNoRow = INT64_MIN;

// A place outside the rows is recorded in the handle's status and moves nothing.
__device__ __forceinline__ void load_picks(const RowsArgs& a, uint64_t t0, int tokens, Picks& s) {
  const uint64_t left = a.tokens - t0;
  const int n = (int)(left < tokens ? left : tokens) * a.top_k;
  for (int i = threadIdx.x; i < tokens * a.top_k; i += blockDim.x) {
    int64_t row = kNoRow;  // tokens past the end have none
    float w = 0.f;
    if (i < n) {
      const uint64_t slot = t0 * a.top_k + i;
      const int64_t p = a.places[slot];
      if ((uint64_t)(p >= 0 ? p : ~p) < a.tokens * (uint64_t)a.top_k) {
        row = p;
        if (p >= 0) w = a.weights ? a.weights[slot] : 1.f;
      } else {
        op_status(a.status, PL_ERR_BOUNDS);
      }
    }
    s.row[i] = row;
    s.w[i] = w;
  }
  __syncthreads();
}

// rows[place_j] = x, for all j: the token is read once.  Bound by DRAM: 8192 x
// 4096 bf16, 8 picks, 92 us, 6.5 TB/s.  SHIFT (rows at any address): 4096 x 2049
// bf16, 8 picks, 32 us, 4.7 TB/s, by 2-byte accesses 65.
template <typename T, bool SHIFT, int U>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(const __grid_constant__ RowsArgs a, int tpt) {
  op_wait();
  __shared__ Picks picks;
  const int per = blockDim.x / tpt, group = threadIdx.x / tpt, lane = threadIdx.x % tpt, k = a.top_k;
  const uint64_t t0 = (uint64_t)blockIdx.x * per * U;
  load_picks(a, t0, per * U, picks);
  constexpr int V = V16<T>;
  const T* x[U];
  bool on[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t t = t0 + u * per + group;
    on[u] = t < a.tokens;
    x[u] = (const T*)a.x + t * a.ldx;
  }
  if (!SHIFT) {
    // every token's vector is read once and stored to all its rows
    for (uint64_t v = lane; v < a.width / V; v += tpt) {
      Pack<T, V> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = ld_row_if<T, false>(x[u] + v * V, on[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) pin(r[u]);
      for (int j = 0; j < k; ++j) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t p = picks.row[(u * per + group) * k + j];
          if (p == kNoRow) continue;
          st_pack_once<T, V>((T*)a.y + (uint64_t)(p >= 0 ? p : ~p) * a.ldy + v * V, p >= 0 ? r[u] : zero_pack<T, V>());
        }
      }
    }
  } else {
    // each row cuts the token its own way; after the first, it is in the L1
#pragma unroll
    for (int u = 0; u < U; ++u) {
      for (int j = 0; j < k; ++j) {
        const int64_t p = picks.row[(u * per + group) * k + j];
        if (p == kNoRow) continue;
        T* y = (T*)a.y + (uint64_t)(p >= 0 ? p : ~p) * a.ldy;
        const Cut c = cut_of<T, true>(y, a.width);
        for (uint64_t v = lane; v < c.nv + c.beside; v += tpt) {
          if (v < c.nv) {
            st_pack_once<T, V>(y + c.head + v * V, ld_row_if<T, true>(x[u] + c.head + v * V, p >= 0));
          } else {
            const uint64_t e = c.at<V>((uint32_t)(v - c.nv));
            y[e] = p >= 0 ? x[u][e] : from_f32<T>(0.f);
          }
        }
      }
    }
  }
}

// y = sum over j of w_j rows[place_j], in binary32, ascending j: J rows of U
// tokens are in flight in each thread.  Four CTAs per SM: with the registers
// that the compiler takes by itself (32), it spreads the loads out again.  Bound
// by DRAM: 8192 x 4096 bf16, 4 / 6 / 8 picks, 52 / 71 / 89 us, 6.5 to 6.8 TB/s.
template <typename T, int U, int J>
__global__ void __launch_bounds__(kRowThreads, 4) combine_kernel(const __grid_constant__ RowsArgs a, int tpt) {
  op_wait();
  __shared__ Picks picks;
  const int per = blockDim.x / tpt, group = threadIdx.x / tpt, lane = threadIdx.x % tpt, k = a.top_k;
  const uint64_t t0 = (uint64_t)blockIdx.x * per * U;
  load_picks(a, t0, per * U, picks);
  constexpr int V = V16<T>;
  for (uint64_t v = lane; v < a.width / V; v += tpt) {
    float acc[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[u][i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += J) {
      Pack<T, V> r[U][J];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int64_t p = j0 + j < k ? picks.row[(u * per + group) * k + j0 + j] : kNoRow;
          r[u][j] = ld_row_if<T, false>((const T*)a.x + (uint64_t)p * a.ldx + v * V, p >= 0);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j) pin(r[u][j]);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float w = j0 + j < k ? picks.w[(u * per + group) * k + j0 + j] : 0.f;  // 0 where nothing was loaded
#pragma unroll
          for (int i = 0; i < V; ++i) acc[u][i] = __fmaf_rn(w, to_f32(r[u][j].v[i]), acc[u][i]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint64_t t = t0 + u * per + group;
      if (t >= a.tokens) continue;
      Pack<T, V> o;
#pragma unroll
      for (int i = 0; i < V; ++i) o.v[i] = from_f32<T>(acc[u][i]);
      st_pack_once<T, V>((T*)a.y + t * a.ldy + v * V, o);
    }
  }
}

// The same for rows that are not 16-byte aligned and short, or in host memory: S
// elements of a thread, tpt apart, of J rows each in flight.  Cutting aligned
// vectors out of the rows' granules moves fewer requests but waits longer for
// each (41 against 25 us for 3001 tokens, 6 rows of 1537 binary32 values).
template <typename T, int S, int J>
__global__ void __launch_bounds__(kRowThreads, 4) combine_narrow_kernel(const __grid_constant__ RowsArgs a, int tpt) {
  op_wait();
  __shared__ Picks picks;
  const int per = blockDim.x / tpt, group = threadIdx.x / tpt, lane = threadIdx.x % tpt, k = a.top_k;
  const uint64_t t0 = (uint64_t)blockIdx.x * per;
  load_picks(a, t0, per, picks);
  for (uint64_t e = lane; e < a.width; e += (uint64_t)S * tpt) {
    float acc[S];
#pragma unroll
    for (int i = 0; i < S; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += J) {
      float x[J][S];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int64_t p = j0 + j < k ? picks.row[group * k + j0 + j] : kNoRow;
        const T* row = (const T*)a.x + (uint64_t)p * a.ldx + e;
#pragma unroll
        for (int i = 0; i < S; ++i) x[j][i] = ld1_if(row + i * tpt, p >= 0 && e + i * tpt < a.width);
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < S; ++i) asm volatile("" : "+f"(x[j][i]));
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float w = j0 + j < k ? picks.w[group * k + j0 + j] : 0.f;
#pragma unroll
        for (int i = 0; i < S; ++i) acc[i] = __fmaf_rn(w, x[j][i], acc[i]);
      }
    }
    if (t0 + group >= a.tokens) continue;
    T* y = (T*)a.y + (t0 + group) * a.ldy + e;
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (e + i * tpt < a.width) y[i * tpt] = from_f32<T>(acc[i]);
  }
}

// The same through shared memory: one CTA for `tile` columns of one token.  Bulk
// copies bring the 16-byte granules that lie whole in each row's piece, at
// the piece's own address modulo 16, and threads the elements beside them, so
// any alignment moves like any other and no registers wait for the rows.  (3001
// tokens of width 1537: 6 picks, binary32, 24.3 us, by registers 25.3; 8 picks,
// bf16, 23.2 against 29.5.  CTAs that stay and fetch the next token's rows during
// the sums were slower, 38 to 46 us: the elements beside the granules then cost a
// round trip in every round.)
constexpr unsigned long long kBulkWaitNs = 2000000000ull;
template <typename T, int J>
__global__ void __launch_bounds__(kRowThreads) combine_bulk_kernel(const __grid_constant__ RowsArgs a, uint32_t tile,
                                                                   uint32_t tiles, uint32_t stride) {
  op_wait();
  extern __shared__ __align__(16) char piece[];  // k pieces, `stride` bytes apart
  __shared__ uint64_t bar;
  __shared__ const T* src[PURLIN_MAX_TOP_K];     // the row's piece, or null
  __shared__ float weight[PURLIN_MAX_TOP_K];
  const int k = a.top_k, tid = threadIdx.x;
  const uint64_t t = blockIdx.x / tiles, c0 = (uint64_t)(blockIdx.x % tiles) * tile;
  const uint32_t n = (uint32_t)min((uint64_t)tile, a.width - c0);
  if (tid < k) {
    const uint64_t slot = t * k + tid;
    const int64_t p = a.places[slot];
    const bool in = (uint64_t)(p >= 0 ? p : ~p) < a.tokens * (uint64_t)k;
    if (!in) op_status(a.status, PL_ERR_BOUNDS);
    const bool live = in && p >= 0;
    src[tid] = live ? (const T*)a.x + (uint64_t)p * a.ldx + c0 : nullptr;
    weight[tid] = live ? (a.weights ? a.weights[slot] : 1.f) : 0.f;
  }
  if (tid == 0) mbar_init(&bar, 1);
  __syncthreads();
  // the granules of a piece: from b0 to b1, offsets from the piece's first byte
  auto first = [](const T* p) { return (uint32_t)(16u - ((uintptr_t)p & 15u)) & 15u; };
  auto last = [n](const T* p) { return (uint32_t)(n * sizeof(T) - (((uintptr_t)p + n * sizeof(T)) & 15u)); };
  if (tid == 0) {
    fence_async_shared();
    fence_async_global();
    uint32_t bytes = 0;
    for (int j = 0; j < k; ++j)
      if (src[j] && n * sizeof(T) >= 32) bytes += last(src[j]) - first(src[j]);
    mbar_expect_tx(&bar, bytes);
    for (int j = 0; j < k; ++j) {
      const T* p = src[j];
      if (!p || n * sizeof(T) < 32) continue;
      const uint32_t b0 = first(p), size = last(p) - b0;  // a multiple of 16, and 16 at least
      bulk_load(piece + (uint64_t)j * stride + ((uintptr_t)p & 15u) + b0, (const char*)p + b0, size, &bar);
    }
  }
  // beside them: fewer than 16 bytes at each end, or all of a short piece
  constexpr int B = 32 / sizeof(T);
  for (int i = tid; i < k * B; i += blockDim.x) {
    const T* p = src[i / B];
    if (!p) continue;
    const uint32_t r = i % B;
    uint32_t e = r;
    bool is = r < n;
    if (n * sizeof(T) >= 32) {
      const uint32_t head = first(p) / sizeof(T), tail = last(p) / sizeof(T);
      e = r < head ? r : tail + r - head;
      is = e < n;
    }
    if (is) ((T*)(piece + (uint64_t)(i / B) * stride + ((uintptr_t)p & 15u)))[e] = p[e];
  }
  if (!__syncthreads_and(mbar_wait(&bar, 0, kBulkWaitNs))) {
    if (tid == 0) op_status(a.status, PL_ERR_TIMEOUT);
    mbar_wait(&bar, 0, kBulkWaitNs);  // the copies in flight still write here
    return;
  }
  T* y = (T*)a.y + t * a.ldy + c0;
  for (int j0 = 0; j0 == 0 || j0 < k; j0 += J) {
    const T* s[J];
    float w[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const bool is = j0 + j < k && src[j0 + j];
      // a dropped pick has no piece and is skipped
      s[j] = is ? (const T*)(piece + (uint64_t)(j0 + j) * stride + ((uintptr_t)src[j0 + j] & 15u)) : nullptr;
      w[j] = is ? weight[j0 + j] : 0.f;
    }
    for (uint32_t e = tid; e < n; e += blockDim.x) {
      float acc = j0 ? ((float*)(piece + (uint64_t)k * stride))[e] : 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (s[j]) acc = __fmaf_rn(w[j], to_f32(s[j][e]), acc);
      if (j0 + J < k) ((float*)(piece + (uint64_t)k * stride))[e] = acc;
      else y[e] = from_f32<T>(acc);
    }
  }
}

// grad_rows[place_j] = w_j dy, grad_w_j = <rows[place_j], dy>: dy is read once
// for J picks, and J rows are in flight in each thread.  The products' parts
// are joined in a fixed order, by lanes and then by warps.  Rows are stored
// evict-first: as ordinary stores they cost a third more.  Bound by DRAM: 8192 x
// 2048 bf16, 6 picks, 69 us, 6.3 TB/s (with 80 registers 75, with 128 94).
template <typename T, int J>
__global__ void __launch_bounds__(kRowThreads, 4) combine_grad_kernel(const __grid_constant__ RowsArgs a, int tpt) {
  op_wait();
  __shared__ Picks picks;
  __shared__ float part[kRowThreads / 32][J];
  const int per = blockDim.x / tpt, group = threadIdx.x / tpt, first = threadIdx.x % tpt, k = a.top_k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t t = (uint64_t)blockIdx.x * per + group;
  load_picks(a, (uint64_t)blockIdx.x * per, per, picks);
  constexpr int V = V16<T>;
  const bool on = t < a.tokens;
  const T* dy = (const T*)a.grad_y + t * a.ldg;
  for (int j0 = 0; j0 < k; j0 += J) {
    float dot[J];
#pragma unroll
    for (int j = 0; j < J; ++j) dot[j] = 0.f;
    for (uint64_t v = first; v < a.width / V; v += tpt) {
      Pack<T, V> g = ld_row_if<T, false>(dy + v * V, on), r[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int64_t p = j0 + j < k ? picks.row[group * k + j0 + j] : kNoRow;
        r[j] = ld_row_if<T, false>((const T*)a.x + (uint64_t)p * a.ldx + v * V, p >= 0);
      }
      pin(g);
#pragma unroll
      for (int j = 0; j < J; ++j) pin(r[j]);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int64_t p = j0 + j < k ? picks.row[group * k + j0 + j] : kNoRow;
        if (p == kNoRow) continue;
        const float w = picks.w[group * k + j0 + j];
        Pack<T, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dot[j] = __fmaf_rn(to_f32(r[j].v[i]), to_f32(g.v[i]), dot[j]);
          o.v[i] = from_f32<T>(w * to_f32(g.v[i]));
        }
        st_pack_once<T, V>((T*)a.y + (uint64_t)(p >= 0 ? p : ~p) * a.ldy + v * V, p >= 0 ? o : zero_pack<T, V>());
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
      for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], d);
      if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (on && first < J && j0 + first < k) {
      float s = 0.f;
      for (int q = 0; q < tpt / 32; ++q) s += part[group * (tpt / 32) + q][first];
      // a dropped pick's row went in as zeros, whose product with an infinite dy is NaN
      a.grad_weights[t * k + j0 + first] = picks.row[group * k + j0 + first] >= 0 ? s : 0.f;
    }
    __syncthreads();
  }
}

// The same for rows that are not 16-byte aligned: one warp for each pick.  3001 x
// 1537 binary32, 6 picks, 57 us, 4.2 TB/s: every granule is asked for twice, and
// more of them in flight only push each other out of the L1 (68 us with four).
template <typename T>
__global__ void __launch_bounds__(kRowThreads) combine_grad_shift_kernel(const __grid_constant__ RowsArgs a) {
  op_wait();
  const uint64_t slot = (uint64_t)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
  if (slot >= a.tokens * a.top_k) return;
  constexpr int V = V16<T>;
  const int lane = threadIdx.x & 31;
  const int32_t p = a.places[slot];
  const bool live = p >= 0;
  const uint64_t row = (uint64_t)(live ? p : ~p);
  if (row >= a.tokens * (uint64_t)a.top_k) {
    if (lane == 0) {
      op_status(a.status, PL_ERR_BOUNDS);
      a.grad_weights[slot] = 0.f;
    }
    return;
  }
  const T* dy = (const T*)a.grad_y + slot / a.top_k * a.ldg;
  const T* x = (const T*)a.x + row * a.ldx;
  T* dx = (T*)a.y + row * a.ldy;
  const float w = live ? a.weights[slot] : 0.f;
  const Cut c = cut_of<T, true>(dx, a.width);
  float dot = 0.f;
  for (uint64_t v = lane; v < c.nv; v += 32) {
    Pack<T, V> g = ld_row_if<T, true>(dy + c.head + v * V, live);
    const Pack<T, V> r = ld_row_if<T, true>(x + c.head + v * V, live);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dot = __fmaf_rn(to_f32(r.v[i]), to_f32(g.v[i]), dot);
      g.v[i] = from_f32<T>(w * to_f32(g.v[i]));
    }
    st_pack_once<T, V>(dx + c.head + v * V, live ? g : zero_pack<T, V>());
  }
  for (uint32_t i = lane; i < c.beside; i += 32) {
    const uint64_t e = c.at<V>(i);
    const float r = ld1_if(x + e, live), g = ld1_if(dy + e, live);
    dot = __fmaf_rn(r, g, dot);
    dx[e] = from_f32<T>(live ? w * g : 0.f);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
  if (lane == 0) a.grad_weights[slot] = dot;
}

// Whether every row is 16-byte aligned and a whole number of vectors.
template <typename T>
bool aligned(const RowsArgs& a) {
  const uint64_t bits = (uint64_t)(uintptr_t)a.x | (uint64_t)(uintptr_t)a.y | (uint64_t)(uintptr_t)a.grad_y |
                        (a.ldx | a.ldy | a.ldg | a.width) * sizeof(T);
  return bits % 16 == 0;
}

}  // namespace

size_t expert_plan_bytes(uint64_t slots, int experts) {
  if (slots <= kClusterSort) return 0;
  return (size_t)(sort_chunks(slots) * (uint64_t)experts * sizeof(uint32_t));
}

purlin_status launch_expert_plan(const PlanArgs& a, cudaStream_t s) {
  const int bins = a.experts + 1;
  purlin_status st;
  if (a.slots <= kClusterSort) {
    const ClusterShape c(a.slots);
    int threads = kClusterThreads;
    if (c.ctas == 1 && c.ipt == 1) {  // few picks: as many warps as they or the bins need
      const uint64_t wide = std::max<uint64_t>(a.slots, bins);
      threads = (int)std::min<uint64_t>(kClusterThreads, (wide + 31) / 32 * 32);
    }
    const size_t smem = (size_t)(threads / 32) * bins * sizeof(uint16_t);
    constexpr int kMost = kClusterThreads / 32 * (kSortBins + 1) * sizeof(uint16_t);
    if ((st = op_smem((const void*)plan_cluster_kernel, smem, kMost))) return st;
    return op_launch_cluster(c.ctas, plan_cluster_kernel, c.ctas, threads, smem, s, a, c.ipt);
  }
  const uint32_t chunk = (uint32_t)sort_chunk(a.slots);
  const uint64_t chunks = sort_chunks(a.slots);
  const size_t smem = (size_t)(kSortThreads / 32) * bins * sizeof(uint16_t);
  if ((st = op_launch(plan_count_kernel, chunks, kSortThreads, 0, s, a, chunk))) return st;
  return op_launch(plan_place_kernel, chunks, kSortThreads, smem, s, a, chunk, (int)(chunk / kSortThreads));
}

template <typename T>
purlin_status dispatch_t(const RowsArgs& a, cudaStream_t s) {
  const bool shift = !aligned<T>(a);
  const RowShape c = RowShape::of<T>(a.width, shift);
  auto go = [&](auto sh, auto u) {
    constexpr int U = decltype(u)::value;
    return op_launch(dispatch_kernel<T, decltype(sh)::value, U>, c.ctas(a.tokens, U), c.tpt * c.per, 0, s, a, c.tpt);
  };
  const std::integral_constant<int, 1> one;
  if (shift) return go(std::true_type(), one);
  // with few copies of each token, two tokens (1 pick: 22 against 24 us at 8192 x 4096; 8 picks: 94 against 92)
  if (a.top_k > 4 || c.ctas(a.tokens, 2) < kManyCtas) return go(std::false_type(), one);
  return go(std::false_type(), std::integral_constant<int, 2>());
}

// f(integral_constant i) for i in 1 .. N
template <int N, typename F>
purlin_status with_int(int i, F f) {
  if constexpr (N > 1)
    if (i < N) return with_int<N - 1>(i, f);
  return f(std::integral_constant<int, N>());
}

// Rows in flight: the picks in as few equal passes of at most 8 as hold them.
int rows_in_flight(int k) {
  const int passes = (k + 7) / 8;
  return (k + passes - 1) / passes;
}

template <typename T>
purlin_status combine_t(const RowsArgs& a, cudaStream_t s) {
  const bool narrow = !aligned<T>(a);
  return with_int<8>(rows_in_flight(a.top_k), [&](auto each) {
    constexpr int J = decltype(each)::value;
    // Long rows in device memory go through shared memory, 40 KiB a CTA (the sums
    // of more than 8 picks take a binary32 row of their own there).  A CTA costs
    // the same for a short row, by registers the time goes with the elements:
    // 8000 tokens, 6 picks: binary32 of 513 columns 34 us, by registers 25; bf16 of
    // 513 columns 32 and 30, of 1025 columns 37 and 47.
    if (narrow && !a.host && a.width >= 768) {
      const uint64_t each = (uint64_t)a.top_k * sizeof(T) + (a.top_k > 8 ? 4 : 0);
      const uint32_t tile = (uint32_t)std::min<uint64_t>(a.width, (40 * 1024 - 32 * a.top_k) / each);
      const uint64_t tiles = (a.width + tile - 1) / tile;
      const uint32_t even = (uint32_t)((a.width + tiles - 1) / tiles);
      const uint32_t stride = (uint32_t)((even * sizeof(T) + 31) & ~(size_t)15);
      const size_t smem = (size_t)stride * a.top_k + (a.top_k > 8 ? (size_t)even * 4 : 0);
      if (purlin_status st = op_smem((const void*)combine_bulk_kernel<T, J>, smem, 48 * 1024)) return st;
      return op_launch(combine_bulk_kernel<T, J>, a.tokens * tiles, kRowThreads, smem, s, a, even, (uint32_t)tiles, stride);
    }
    if (narrow) {
      constexpr int S = sizeof(T) == 4 ? 2 : 4;
      const RowShape c((a.width + S - 1) / S);
      return op_launch(combine_narrow_kernel<T, S, J>, c.ctas(a.tokens, 1), c.tpt * c.per, 0, s, a, c.tpt);
    }
    // with few picks, more tokens
    constexpr int U = J == 1 ? 4 : J == 2 ? 2 : 1;
    const RowShape c(a.width / V16<T>);
    if (U > 1 && c.ctas(a.tokens, U) >= kManyCtas)
      return op_launch(combine_kernel<T, U, J>, c.ctas(a.tokens, U), c.tpt * c.per, 0, s, a, c.tpt);
    return op_launch(combine_kernel<T, 1, J>, c.ctas(a.tokens, 1), c.tpt * c.per, 0, s, a, c.tpt);
  });
}

template <typename T>
purlin_status combine_grad_t(const RowsArgs& a, cudaStream_t s) {
  if (!aligned<T>(a)) {
    const uint64_t grid = (a.tokens * a.top_k + kRowThreads / 32 - 1) / (kRowThreads / 32);
    return op_launch(combine_grad_shift_kernel<T>, grid, kRowThreads, 0, s, a);
  }
  return with_int<8>(rows_in_flight(a.top_k), [&](auto each) {
    const RowShape c(a.width / V16<T>);
    return op_launch(combine_grad_kernel<T, decltype(each)::value>, c.ctas(a.tokens, 1), c.tpt * c.per, 0, s, a, c.tpt);
  });
}

purlin_status launch_dispatch(const RowsArgs& a, int dtype, cudaStream_t s) {
  return dtype == PL_F32 ? dispatch_t<float>(a, s) : dispatch_t<bf16>(a, s);
}
purlin_status launch_combine(const RowsArgs& a, int dtype, cudaStream_t s) {
  return dtype == PL_F32 ? combine_t<float>(a, s) : combine_t<bf16>(a, s);
}
purlin_status launch_combine_grad(const RowsArgs& a, int dtype, cudaStream_t s) {
  return dtype == PL_F32 ? combine_grad_t<float>(a, s) : combine_grad_t<bf16>(a, s);
}

}  // namespace pl
