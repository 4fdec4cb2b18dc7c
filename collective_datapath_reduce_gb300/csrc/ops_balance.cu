// The balance of the experts' load: how often each was picked and what share of
// the tokens' scores it has, the loss that couples the two, and its gradient.
#include <math.h>

#include <type_traits>

#include "ops_common.cuh"

namespace pl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 16;           // of a CTA, a token each at a time
constexpr int kThreads = kWarps * 32;
constexpr int kMostCtas = 2 * 152;   // that leave sums
constexpr int kRows = 8;             // warps whose sums have a row of shared memory
constexpr int kCluster = 8;          // CTAs whose sums are added through shared memory

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}
// Largest value of the warp, NaN the lesser of any two.
__device__ __forceinline__ float redux_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// A word of the shared memory of the cluster's CTA `rank`, where p is in this one's.
__device__ __forceinline__ uint32_t ld_cluster(const void* p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// A row's values in a warp's lanes, N (an even number) in each: vectors of M
// neighbours, 32 vectors apart, or single values where the row is not made of such.
template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Lane {
  static constexpr int M = N * sizeof(T) > 16 ? 16 / sizeof(T) : N;
  T v[N];
  // Which value the lane's i-th is.
  static __device__ __forceinline__ int at(int i, bool vec) {
    const int lane = threadIdx.x & 31;
    return vec ? (lane + i / M * 32) * M + i % M : lane + i * 32;
  }
  // The row at p; values past its width are `none`.
  __device__ __forceinline__ void load(const T* p, int width, bool vec, float none) {
    if (vec) {
#pragma unroll
      for (int q = 0; q < N; q += M) {
        Pack<T, M> r;
        if (at(q, true) < width) r = *reinterpret_cast<const Pack<T, M>*>(p + at(q, true));
        else
#pragma unroll
          for (int i = 0; i < M; ++i) r.v[i] = from_f32<T>(none);
#pragma unroll
        for (int i = 0; i < M; ++i) v[q + i] = r.v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = at(i, false) < width ? p[at(i, false)] : from_f32<T>(none);
    }
  }
  __device__ __forceinline__ void store(T* p, int width, bool vec) const {
    if (vec) {
#pragma unroll
      for (int q = 0; q < N; q += M) {
        Pack<T, M> r;
#pragma unroll
        for (int i = 0; i < M; ++i) r.v[i] = v[q + i];
        if (at(q, true) < width) st_pack(p + at(q, true), r);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (at(i, false) < width) p[at(i, false)] = v[i];
    }
  }
  __device__ __forceinline__ void pairs(F2 (&p)[N / 2]) const {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) p[i] = f2(to_f32(v[2 * i]), to_f32(v[2 * i + 1]));
  }
  __device__ __forceinline__ void round(const F2 (&p)[N / 2]) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 of = split(p[i]);
      v[2 * i] = from_f32<T>(of.x);
      v[2 * i + 1] = from_f32<T>(of.y);
    }
  }
};

// 2^x; results below the smallest normal number are 0.
__device__ __forceinline__ F2 ex2(F2 x) {
  float2 s = split(x);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(s.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(s.y));
  return f2(s.x, s.y);
}
// 1 / x, within 1 ulp; of a number past 2^126, 0.
__device__ __forceinline__ F2 inverse(F2 x) {
  float2 s = split(x);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(s.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(s.y));
  return f2(s.x, s.y);
}

// The lesser of two values, NaN if one of them is.
__device__ __forceinline__ float lesser(float x, float y) {
  float m;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(x), "f"(y));
  return m;
}

// A token's logits become its scores as shares of one, x; `slope` is what a
// score's derivative has beside them, 1 - sigmoid = exp(-logit) x sigmoid.  A row
// of nothing but -inf has shares of 0.  No decision hangs on them, so neither
// exponentials nor reciprocals need be the nearest numbers.
constexpr float kLog2e = 1.4426950408889634f;
template <typename T, int N>
__device__ __forceinline__ void shares(const Lane<T, N>& row, int sigmoid, F2 (&x)[N / 2], F2 (&slope)[N / 2]) {
  constexpr int P = N / 2;
  F2 sum = f2(0.f);
  float s;
  row.pairs(x);
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      // exp(-x) at most 2^127: a sigmoid below 2^-126 is 0, and the slope a number, of NaN neither
      const float2 a = split(x[i] * f2(-kLog2e));
      const F2 e = ex2(f2(lesser(a.x, 127.f), lesser(a.y, 127.f)));
      x[i] = inverse(f2(1.f) + e);
      slope[i] = e * x[i];
      sum = sum + x[i];
    }
    s = warp_sum(both(sum)) + 1e-20f;
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 a = split(x[i]);
      m = fmaxf(m, fmaxf(a.x, a.y));
    }
    m = redux_max(m);
    if (m == -INFINITY) m = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      x[i] = ex2((x[i] + f2(-m)) * f2(kLog2e));
      slope[i] = f2(1.f);
      sum = sum + x[i];
    }
    s = warp_sum(both(sum));
    if (s == 0.f) s = 1.f;
  }
  s = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = x[i] * f2(s);
}

// The loss of picks C, shares P and N tokens: scale x E x sum C P / (sum C x N).
__device__ __forceinline__ float loss_of(const BalanceArgs& a, float picks, float dot, float tokens) {
  const float all = picks * tokens;
  return all > 0.f ? a.scale * (float)a.experts * __fdiv_rn(dot, all) : 0.f;
}

// The threads of this CTA, of a cluster's, take experts first .. first + per, at(e)
// being an expert's picks (as bits) and shares, and `tokens` the tokens: they
// write the outputs.  tmp: two words for each warp.
template <typename A>
__device__ __forceinline__ void finish(const BalanceArgs& a, float tokens, float* tmp, int first, int per, A at) {
  const uint32_t rank = cluster_rank();
  float picks = 0.f, dot = 0.f;
  const int e = first + threadIdx.x;
  if ((int)threadIdx.x < per && e < a.experts) {
    const float2 v = at(e);
    const uint32_t c = __float_as_uint(v.x);
    const float p = v.y;
    a.counts[e] = (int32_t)c;
    a.sums[e] = (float)c;
    a.sums[a.experts + e] = p;
    picks = (float)c;
    dot = (float)c * p;
  }
  if (rank == 0 && threadIdx.x == 0) a.sums[2 * a.experts] = tokens;
  if (!a.loss) return;
  picks = warp_sum(picks);
  dot = warp_sum(dot);
  if ((threadIdx.x & 31) == 0) {
    tmp[threadIdx.x >> 5] = picks;
    tmp[kWarps + (threadIdx.x >> 5)] = dot;
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x < 32) {
    picks = dot = 0.f;
#pragma unroll
    for (int i = threadIdx.x; i < kCluster * kWarps; i += 32) {
      picks += __uint_as_float(ld_cluster(tmp + i % kWarps, i / kWarps));
      dot += __uint_as_float(ld_cluster(tmp + kWarps + i % kWarps, i / kWarps));
    }
    picks = warp_sum(picks);
    dot = warp_sum(dot);
    if (threadIdx.x == 0) *a.loss = loss_of(a, picks, dot, tokens);
  }
  cluster_sync();  // before a CTA ends whose memory is read
}

// A token of a warp: its picks, one in each of the first lanes, and its logits.
// Fetched a token ahead: padding's logits are loaded too, and not used.
template <typename T, int N>
struct Token {
  int id;
  Lane<T, N> row;
  __device__ __forceinline__ void load(const BalanceArgs& a, uint64_t t, int vec) {
    const int lane = threadIdx.x & 31;
    id = lane < a.top_k ? a.ids[t * a.top_k + lane] : -1;
    row.load((const T*)a.logits + t * a.ld, a.experts, vec, -INFINITY);
  }
};

// A warp holds a token, N experts in each lane, and adds its
// shares to the lane's sums; picks are counted in shared memory.  The warps'
// sums are added in order, then, of one cluster `alone`, the CTAs'.
//
// Bound by the chain of a token (its loads, exponentials, two reductions across
// the warp), of which an SM has 32 at once: 65536 x 256 binary32, sigmoid, 8 picks take 17.7
// us, 61% of the issue slots and 3.9 TB/s (the logits alone: 9.9 us).  60 us with 16
// warps an SM that load a token when they need it, 30 with 32 and a token fetched
// ahead, 16 to 18 with two values an instruction and no clusters, which left SMs
// without CTAs.  Fetching two tokens ahead (20.4 against 19.0 us with the second
// kernel), CTAs of 32 warps (25.8) and three CTAs an SM (23) were slower.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads, N > 16 ? 1 : 2) balance_kernel(const __grid_constant__ BalanceArgs a, int vec, int alone) {
  op_wait();
  extern __shared__ float dyn[];   // [kRows][experts] shares, whose first row the CTA's become; [experts] picks
  __shared__ uint32_t tokens_of[kWarps];
  __shared__ float tmp[2 * kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts;
  uint32_t* picks = (uint32_t*)(dyn + kRows * E);
  const uint64_t step = (uint64_t)gridDim.x * kWarps;
  // a cluster's CTAs take neighbouring tokens, warp by warp
  uint64_t t = (uint64_t)blockIdx.x * kWarps + warp;
  Token<T, N> now, next;
  constexpr bool AHEAD = N <= 16;  // the registers of a token more
  if (AHEAD && t < a.tokens) next.load(a, t, vec);
  for (int e = threadIdx.x; e < E; e += kThreads) picks[e] = 0;
  __syncthreads();
  constexpr int P = N / 2;
  F2 sum[P];
#pragma unroll
  for (int i = 0; i < P; ++i) sum[i] = f2(0.f);
  uint32_t counted = 0;
  for (; t < a.tokens; t += step) {
    if constexpr (AHEAD) {
      now = next;
      if (t + step < a.tokens) next.load(a, t + step, vec);
    } else {
      now.load(a, t, vec);
    }
    const bool on = now.id >= 0 && now.id < E;
    if (!__any_sync(kAll, on)) continue;  // padding: its logits may be anything
    if (on) atomicAdd(picks + now.id, 1u);
    F2 x[P], slope[P];
    shares<T, N>(now.row, a.sigmoid, x, slope);
#pragma unroll
    for (int i = 0; i < P; ++i) sum[i] = sum[i] + x[i];
    ++counted;
  }
  if (lane == 0) tokens_of[warp] = counted;
  // kRows warps at a time: the next ones add to what those before them left
  for (int first = 0; first < kWarps; first += kRows) {
    if (warp / kRows == first / kRows)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = Lane<T, N>::at(i, vec);
        const float2 of = split(sum[i / 2]);
        if (e < E) dyn[warp % kRows * E + e] = (i % 2 ? of.y : of.x) + (first ? dyn[warp % kRows * E + e] : 0.f);
      }
    __syncthreads();
  }
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float s = dyn[e];
#pragma unroll
    for (int w = 1; w < kRows; ++w) s += dyn[w * E + e];
    dyn[e] = s;
  }
  if (!alone) {  // this CTA's sums are for balance_parts_kernel
    uint32_t* out = a.parts + (uint64_t)blockIdx.x * (2 * E + 1);
    for (int e = threadIdx.x; e < E; e += kThreads) {
      out[e] = picks[e];
      out[E + e] = __float_as_uint(dyn[e]);
    }
    if (threadIdx.x == 0) {
      uint32_t tokens = 0;
      for (int w = 0; w < kWarps; ++w) tokens += tokens_of[w];
      out[2 * E] = tokens;
    }
    return;
  }
  cluster_sync();
  uint32_t tokens = 0;
  for (int i = lane; i < kCluster * kWarps; i += 32) tokens += ld_cluster(tokens_of + i % kWarps, i / kWarps);
  tokens = __reduce_add_sync(kAll, tokens);
  const int per = (E + kCluster - 1) / kCluster;
  finish(a, (float)tokens, tmp, (int)cluster_rank() * per, per, [&](int e) {
    uint32_t c = 0;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) {
      c += ld_cluster(picks + e, r);
      s += __uint_as_float(ld_cluster(dyn + e, r));
    }
    return make_float2(__uint_as_float(c), s);
  });
  cluster_sync();
}

// The CTAs' sums (304 of them behind a large batch, 620 KB: about 4 us, two round trips
// to the L2 and two cluster barriers): a cluster whose CTAs take `per` neighbouring experts each, in
// up to 32 threads each that share the CTAs' sums and are added in order.
__global__ void __launch_bounds__(kThreads) balance_parts_kernel(const __grid_constant__ BalanceArgs a, int ctas, int per) {
  op_wait();
  __shared__ float tmp[2 * kWarps];
  __shared__ float sum[kThreads];
  __shared__ uint32_t picks[kThreads];
  const int E = a.experts, row = 2 * E + 1, first = (int)cluster_rank() * per;
  uint32_t tokens = 0;
  for (int p = threadIdx.x & 31; p < ctas; p += 32) tokens += a.parts[(uint64_t)p * row + 2 * E];
  const int columns = min(kThreads / per, 32), e = first + threadIdx.x % per;
  uint32_t c = 0;
  float s = 0.f;
  if (e < E && (int)threadIdx.x < columns * per) {
#pragma unroll 8
    for (int p = threadIdx.x / per; p < ctas; p += columns) {
      c += a.parts[(uint64_t)p * row + e];
      s += __uint_as_float(a.parts[(uint64_t)p * row + E + e]);
    }
  }
  picks[threadIdx.x] = c;
  sum[threadIdx.x] = s;
  tokens = __reduce_add_sync(kAll, tokens);
  __syncthreads();
  finish(a, (float)tokens, tmp, first, per, [&](int e) {
    uint32_t c = 0;
    float s = 0.f;
    for (int q = 0; q < columns; ++q) {
      c += picks[q * per + e - first];
      s += sum[q * per + e - first];
    }
    return make_float2(__uint_as_float(c), s);
  });
  cluster_sync();
}

// The sum of the picks that `sums` hold, in every thread of the CTA.
__device__ __forceinline__ float all_picks(const float* sums, int experts, float* tmp) {
  float s = 0.f;
  for (int e = threadIdx.x; e < experts; e += kThreads) s += sums[e];
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = s;
  __syncthreads();
  s = tmp[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) s += tmp[w];
  return s;
}

__global__ void __launch_bounds__(kThreads) balance_join_kernel(const __grid_constant__ BalanceArgs a) {
  op_wait();
  __shared__ float tmp[2][kWarps];
  const float picks = all_picks(a.sums, a.experts, tmp[0]);
  float dot = 0.f;
  for (int e = threadIdx.x; e < a.experts; e += kThreads) dot = __fmaf_rn(a.sums[e], a.sums[a.experts + e], dot);
  dot = warp_sum(dot);
  if ((threadIdx.x & 31) == 0) tmp[1][threadIdx.x >> 5] = dot;
  __syncthreads();
  dot = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) dot += tmp[1][w];
  if (threadIdx.x == 0) *a.loss = loss_of(a, picks, dot, a.sums[2 * a.experts]);
}

// With p the shares and c_e = dL x scale x E x C_e / (sum C x N):  dx_j = p_j (c_j -
// sum p c), for sigmoids times 1 - s_j.  A token without picks has none.
//
// 65536 x 256 binary32 run at 5.7 TB/s (23.9 us); small batches wait for the CTAs' first round
// trips, the sums' and the tokens' (16383 x 160 bf16 on a base: 7.9 us, of which 2.4 are
// the bytes').
template <typename T, int N>
__global__ void __launch_bounds__(kThreads, N > 8 ? 1 : 2) balance_grad_kernel(const __grid_constant__ BalanceArgs a, int vec) {
  op_wait();
  __shared__ float tmp[kWarps];
  const int warp = threadIdx.x >> 5, E = a.experts;
  const uint64_t step = (uint64_t)gridDim.x * kWarps;
  uint64_t t = (uint64_t)blockIdx.x * kWarps + warp;
  Token<T, N> now, next;
  Lane<T, N> base, next_base;
  constexpr bool AHEAD = N <= 16;  // the registers of a token more
  if (AHEAD && t < a.tokens) {
    next.load(a, t, vec);
    if (a.base) next_base.load((const T*)a.base + t * a.ldb, E, vec, 0.f);
  }
  const float all = all_picks(a.sums, E, tmp) * a.sums[2 * E];
  const float f = all > 0.f ? __fdiv_rn((a.grad_loss ? *a.grad_loss : 1.f) * a.scale * (float)E, all) : 0.f;
  constexpr int P = N / 2;
  F2 c[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = Lane<T, N>::at(2 * i, vec), o = Lane<T, N>::at(2 * i + 1, vec);
    c[i] = f2(f) * f2(e < E ? a.sums[e] : 0.f, o < E ? a.sums[o] : 0.f);
  }
  for (; t < a.tokens; t += step) {
    if constexpr (AHEAD) {
      now = next;
      base = next_base;
      if (t + step < a.tokens) {
        next.load(a, t + step, vec);
        if (a.base) next_base.load((const T*)a.base + (t + step) * a.ldb, E, vec, 0.f);
      }
    } else {
      now.load(a, t, vec);
    }
    F2 x[P], slope[P];
    if (__any_sync(kAll, now.id >= 0 && now.id < E)) {
      shares<T, N>(now.row, a.sigmoid, x, slope);
      F2 sum = f2(0.f);
#pragma unroll
      for (int i = 0; i < P; ++i) sum = fma2(x[i], c[i], sum);
      const float dot = warp_sum(both(sum));
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = x[i] * (c[i] + f2(-dot)) * slope[i];
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = f2(0.f);
    }
    if (a.base) {
      if (!AHEAD) base.load((const T*)a.base + t * a.ldb, E, vec, 0.f);
      base.pairs(slope);
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = x[i] + slope[i];
    }
    now.row.round(x);
    now.row.store((T*)a.grad_logits + t * a.ldg, E, vec);
  }
}

// Experts of a lane: the smallest power of two, 2 at least, that covers them with 32 lanes.
template <typename F>
purlin_status with_lanes(int experts, F f) {
  if (experts <= 64) return f(std::integral_constant<int, 2>());
  if (experts <= 128) return f(std::integral_constant<int, 4>());
  if (experts <= 256) return f(std::integral_constant<int, 8>());
  if (experts <= 512) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

template <typename T, int N>
bool even(const BalanceArgs& a) {
  constexpr uint64_t need = Lane<T, N>::M * sizeof(T);
  uint64_t bits = (uint64_t)(uintptr_t)a.logits | a.ld * sizeof(T);
  if (a.grad_logits) bits |= (uint64_t)(uintptr_t)a.grad_logits | a.ldg * sizeof(T);
  if (a.base) bits |= (uint64_t)(uintptr_t)a.base | a.ldb * sizeof(T);
  return a.experts % Lane<T, N>::M == 0 && bits % need == 0;  // a vector's experts exist or none
}

// Few tokens go through one cluster and one launch, 16 for each of its warps at
// most: the second launch costs the host 3 us (calls of 1000 x 256 / 2000 x 256 / 2000 x 500: 10.5 / 11.0 /
// 15.3 us in one launch, 13.5 / 13.4 / 13.6 in two; on the device 7.7 / 11.0 / 15.3 and 7.1 / 8.7 / 10.8).
bool few(uint64_t tokens, int experts) {
  return tokens <= kCluster * kWarps * 16 && tokens * (uint64_t)experts <= kCluster * kWarps * 16 * 256;
}
int ctas_of(uint64_t tokens, int experts) {
  return few(tokens, experts) ? kCluster : (int)std::min<uint64_t>(kMostCtas, (tokens + kWarps - 1) / kWarps);
}

}  // namespace

// The sums of the CTAs of two launches, asked for past 512 tokens whichever way a call
// then goes.
size_t balance_bytes(uint64_t tokens, int experts) {
  const uint64_t ctas = std::min<uint64_t>(kMostCtas, (tokens + kWarps - 1) / kWarps);
  return tokens <= kCluster * kWarps * 4 ? 0 : (size_t)ctas * (2 * (size_t)experts + 1) * sizeof(uint32_t);
}

purlin_status launch_balance(const BalanceArgs& a, int dtype, cudaStream_t s) {
  const bool alone = few(a.tokens, a.experts);
  const int ctas = ctas_of(a.tokens, a.experts), per = (a.experts + kCluster - 1) / kCluster;
  const size_t smem = (size_t)(kRows + 1) * a.experts * sizeof(float);
  const purlin_status st = with_lanes(a.experts, [&](auto n) {
    constexpr int N = decltype(n)::value;
    const int c = alone ? kCluster : 1;
    if (dtype == PL_F32) return op_launch_cluster(c, balance_kernel<float, N>, ctas, kThreads, smem, s, a, (int)even<float, N>(a), (int)alone);
    return op_launch_cluster(c, balance_kernel<bf16, N>, ctas, kThreads, smem, s, a, (int)even<bf16, N>(a), (int)alone);
  });
  if (st || alone) return st;
  return op_launch_cluster(kCluster, balance_parts_kernel, kCluster, kThreads, 0, s, a, ctas, per);
}

purlin_status launch_balance_join(const BalanceArgs& a, cudaStream_t s) {
  return op_launch(balance_join_kernel, 1, kThreads, 0, s, a);
}

purlin_status launch_balance_grad(const BalanceArgs& a, int dtype, cudaStream_t s) {
  const uint64_t grid = std::min<uint64_t>((a.tokens + kWarps - 1) / kWarps, 152 * 2);
  return with_lanes(a.experts, [&](auto n) {
    constexpr int N = decltype(n)::value;
    if (dtype == PL_F32) return op_launch(balance_grad_kernel<float, N>, grid, kThreads, 0, s, a, (int)even<float, N>(a));
    return op_launch(balance_grad_kernel<bf16, N>, grid, kThreads, 0, s, a, (int)even<bf16, N>(a));
  });
}

}  // namespace pl
