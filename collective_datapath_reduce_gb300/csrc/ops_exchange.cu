// The exchange of token rows with experts: the plan (a stable sort of the
// picks by expert), the copy of rows by it, the weighted sum back, and the
// sum's gradient.  The copies are a copy Atom whose destinations are named by
// index, the sum an N-to-1 reduce Atom whose sources are.
#include <type_traits>

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

__global__ void __launch_bounds__(kSortThreads) plan_count_kernel(const __grid_constant__ PlanArgs a, uint32_t chunk) {
  op_wait();
  __shared__ uint32_t hist[kSortBins + 1];
  const int bins = a.experts + 1;
  for (int b = threadIdx.x; b < bins; b += blockDim.x) hist[b] = 0;
  __syncthreads();
  const uint64_t i0 = (uint64_t)blockIdx.x * chunk;
  for (uint32_t i = threadIdx.x; i < chunk; i += blockDim.x) {
    const int e = expert_of(a.ids, i0 + i, a.slots, a.experts);
    if (e >= 0) atomicAdd(hist + e, 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += blockDim.x) a.counts[(uint64_t)blockIdx.x * bins + b] = hist[b];
}

// One chunk's places.  counts == nullptr: the chunk is everything.
__global__ void __launch_bounds__(kSortThreads) plan_place_kernel(const __grid_constant__ PlanArgs a, uint32_t chunk,
                                                                  int ipt) {
  op_wait();
  extern __shared__ uint16_t cnt[];
  __shared__ uint32_t base[kSortBins + 1], before[kSortBins + 1], tmp[33];
  const int bins = a.experts + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t i0 = (uint64_t)blockIdx.x * chunk;
  int digit[kSortIpt];
  uint32_t local[kSortIpt];
#pragma unroll
  for (int q = 0; q < kSortIpt; ++q)
    if (q < ipt) digit[q] = expert_of(a.ids, i0 + (uint64_t)(warp * ipt + q) * 32 + lane, a.slots, a.experts);
  if (a.counts) {
    sum_chunks(a.counts, gridDim.x, blockIdx.x, bins, base, before);
    rank_chunk(digit, local, ipt, bins, cnt, [](int, uint32_t) {});
  } else {
    rank_chunk(digit, local, ipt, bins, cnt, [&](int b, uint32_t n) {
      base[b] = n;
      before[b] = 0;
    });
  }
  uint32_t carry = 0;
  for (int b0 = 0; b0 < a.experts; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    const uint32_t n = b < a.experts ? base[b] : 0;
    uint32_t total;
    const uint32_t at = carry + block_exclusive(n, tmp, &total);
    if (b < a.experts) {
      base[b] = at + before[b];
      if (blockIdx.x == 0) a.offsets[b] = (int32_t)at;
    }
    carry += total;
  }
  if (threadIdx.x == 0) {
    base[a.experts] = carry + before[a.experts];
    if (blockIdx.x == 0) a.offsets[a.experts] = (int32_t)carry;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kSortIpt; ++q) {
    if (q < ipt && digit[q] >= 0) {
      const uint64_t i = i0 + (uint64_t)(warp * ipt + q) * 32 + lane;
      const int32_t p = (int32_t)(base[digit[q]] + cnt[warp * bins + digit[q]] + local[q]);
      a.places[i] = digit[q] == a.experts ? ~p : p;
    }
  }
}

// ------------------------------------------------------------ rows by index

constexpr int kRowThreads = 256;

// A token's row by `tpt` neighbouring threads, 256 / tpt tokens in a CTA.
struct Lane {
  uint64_t token;
  uint32_t first, step;
};

__device__ __forceinline__ Lane lane_of(int tpt) {
  return {(uint64_t)blockIdx.x * (kRowThreads / tpt) + threadIdx.x / tpt, threadIdx.x % tpt, (uint32_t)tpt};
}

// Row of a pick in [0, rows), and whether the pick is live (~row: dropped).  A
// place outside is recorded in the handle's status and moves nothing.
__device__ __forceinline__ bool row_of(const RowsArgs& a, uint64_t slot, uint64_t* row, bool* live) {
  const int32_t p = a.places[slot];
  *live = p >= 0;
  *row = (uint64_t)(p >= 0 ? p : ~p);
  if (*row < a.tokens * (uint64_t)a.top_k) return true;
  op_status(a.status, PL_ERR_BOUNDS);
  *live = false;
  return false;
}

template <typename T, int N>
__global__ void __launch_bounds__(kRowThreads) dispatch_kernel(const __grid_constant__ RowsArgs a, int tpt) {
  op_wait();
  const Lane l = lane_of(tpt);
  if (l.token >= a.tokens) return;
  const T* x = (const T*)a.x + l.token * a.ldx;
  const uint64_t nv = a.width / N;
  for (uint64_t v = l.first; v < nv; v += l.step) {
    const Pack<T, N> r = ld_pack<T, N>(x + v * N);
    for (int j = 0; j < a.top_k; ++j) {
      uint64_t row;
      bool live;
      if (!row_of(a, l.token * a.top_k + j, &row, &live)) continue;
      st_pack<T, N>((T*)a.y + row * a.ldy + v * N, live ? r : zero_pack<T, N>());
    }
  }
}

// y = sum over j of w_j rows[place_j], in binary32, ascending j.
template <typename T, int N>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(const __grid_constant__ RowsArgs a, int tpt) {
  op_wait();
  const Lane l = lane_of(tpt);
  if (l.token >= a.tokens) return;
  T* y = (T*)a.y + l.token * a.ldy;
  const uint64_t nv = a.width / N;
  for (uint64_t v = l.first; v < nv; v += l.step) {
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int j = 0; j < a.top_k; ++j) {
      uint64_t row;
      bool live;
      if (!row_of(a, l.token * a.top_k + j, &row, &live) || !live) continue;
      const float w = a.weights ? a.weights[l.token * a.top_k + j] : 1.f;
      const Pack<T, N> r = ld_pack<T, N>((const T*)a.x + row * a.ldx + v * N);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = __fmaf_rn(w, to_f32(r.v[i]), acc[i]);
    }
    Pack<T, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f32<T>(acc[i]);
    st_pack<T, N>(y + v * N, o);
  }
}

// grad_rows[place_j] = w_j dy, grad_w_j = <rows[place_j], dy>: one warp per
// token and pick holds the product's partial sums.
template <typename T, int N>
__global__ void __launch_bounds__(kRowThreads) combine_grad_kernel(const __grid_constant__ RowsArgs a) {
  op_wait();
  const uint64_t slot = (uint64_t)blockIdx.x * (kRowThreads / 32) + threadIdx.x / 32;
  if (slot >= a.tokens * a.top_k) return;
  const int lane = threadIdx.x & 31;
  uint64_t row;
  bool live;
  const bool in = row_of(a, slot, &row, &live);
  const float w = a.weights && live ? a.weights[slot] : live ? 1.f : 0.f;
  const T* dy = (const T*)a.grad_y + slot / a.top_k * a.ldg;
  const T* x = (const T*)a.x + row * a.ldx;
  T* dx = (T*)a.y + row * a.ldy;
  float dot = 0.f;
  if (in) {
    const uint64_t nv = a.width / N;
#pragma unroll 2
    for (uint64_t v = lane; v < nv; v += 32) {
      const Pack<T, N> g = ld_pack<T, N>(dy + v * N);
      Pack<T, N> o = zero_pack<T, N>();
      if (live) {
        const Pack<T, N> r = ld_pack<T, N>(x + v * N);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dot = __fmaf_rn(to_f32(r.v[i]), to_f32(g.v[i]), dot);
          o.v[i] = from_f32<T>(w * to_f32(g.v[i]));
        }
      }
      st_pack<T, N>(dx + v * N, o);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
  if (lane == 0) a.grad_weights[slot] = dot;
}

template <typename T>
uint64_t row_bits(const RowsArgs& a) {
  return (uint64_t)(uintptr_t)a.x | (uint64_t)(uintptr_t)a.y | (uint64_t)(uintptr_t)a.grad_y |
         (a.ldx | a.ldy | a.ldg | a.width) * sizeof(T);
}

// Threads per token: a power of two that covers the row, 32 to 256.
int threads_per_token(uint64_t nv) {
  int t = 32;
  while (t < kRowThreads && (uint64_t)t < nv) t *= 2;
  return t;
}

}  // namespace

size_t expert_plan_bytes(uint64_t slots, int experts) {
  if (slots <= kSortSmall) return 0;
  return (size_t)(sort_chunks(slots) * (uint64_t)(experts + 1) * sizeof(uint32_t));
}

purlin_status launch_expert_plan(const PlanArgs& in, cudaStream_t s) {
  PlanArgs a = in;
  const int bins = a.experts + 1;
  static_assert(kSortWarps * (kSortBins + 1) * sizeof(uint16_t) <= 96 * 1024, "counters fit shared memory");
  const cudaError_t e = cudaFuncSetAttribute(plan_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return PL_ERR_CUDA;
  }
  if (a.slots <= kSortSmall) {
    a.counts = nullptr;
    const int ipt = (int)std::max<uint64_t>(1, (a.slots + kSortThreads - 1) / kSortThreads);
    const int threads = (int)std::min<uint64_t>(kSortThreads, std::max<uint64_t>(32, (std::max<uint64_t>(a.slots, bins) + 31) / 32 * 32));
    return op_launch(plan_place_kernel, 1, threads, (size_t)(threads / 32) * bins * sizeof(uint16_t), s, a, (uint32_t)0, ipt);
  }
  const uint64_t chunk = sort_chunk(a.slots);
  if (purlin_status st = op_launch(plan_count_kernel, sort_chunks(a.slots), kSortThreads, 0, s, a, (uint32_t)chunk)) return st;
  return op_launch(plan_place_kernel, sort_chunks(a.slots), kSortThreads, (size_t)kSortWarps * bins * sizeof(uint16_t), s, a,
                   (uint32_t)chunk, (int)(chunk / kSortThreads));
}

template <typename T>
purlin_status dispatch_t(const RowsArgs& a, cudaStream_t s) {
  return with_vec<T>(vec_bytes(row_bits<T>(a)), [&](auto n) {
    constexpr int N = decltype(n)::value;
    const int tpt = threads_per_token(a.width / N);
    return op_launch(dispatch_kernel<T, N>, (a.tokens + kRowThreads / tpt - 1) / (kRowThreads / tpt), kRowThreads, 0, s, a, tpt);
  });
}

template <typename T>
purlin_status combine_t(const RowsArgs& a, cudaStream_t s) {
  return with_vec<T>(vec_bytes(row_bits<T>(a)), [&](auto n) {
    constexpr int N = decltype(n)::value;
    const int tpt = threads_per_token(a.width / N);
    return op_launch(combine_kernel<T, N>, (a.tokens + kRowThreads / tpt - 1) / (kRowThreads / tpt), kRowThreads, 0, s, a, tpt);
  });
}

template <typename T>
purlin_status combine_grad_t(const RowsArgs& a, cudaStream_t s) {
  return with_vec<T>(vec_bytes(row_bits<T>(a)), [&](auto n) {
    constexpr int N = decltype(n)::value;
    return op_launch(combine_grad_kernel<T, N>, (a.tokens * a.top_k + kRowThreads / 32 - 1) / (kRowThreads / 32), kRowThreads, 0,
                     s, a);
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
