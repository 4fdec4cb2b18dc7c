// Distillation from a teacher's top logits: the Kullback-Leibler divergence of a
// token's distribution over the vocabulary from the teacher's over its picks,
// and its gradient, over the whole vocabulary or a rank's range of it.
//
// With z the logits, t the teacher's, both over the temperature, q = softmax(t)
// over the picks and p = softmax(z) over the vocabulary, the loss is sum q_k (log q_k
// - log p_k).  A range gives m = max z, s = sum exp(z - m), c = the sum over its
// picks of q_k (log q_k - (z_k - m)), and Q, the sum of their q_k; then, with M
// and S those of all ranges, the loss is the sum of c_r - Q_r (m_r - M) + Q_r log S.
// Differences from the maximum are taken before anything is scaled, so that rows
// of the lowest value are rows like others.
#include <math.h>

#include <type_traits>

#include "ops_common.cuh"

namespace pl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kMostCluster = 8;    // CTAs of a token

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster(const void* p, uint32_t rank, float2 v) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

// 2^x; results below the smallest normal number are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ F2 ex2(F2 x) {
  const float2 s = split(x);
  return f2(ex2(s.x), ex2(s.y));
}

// The largest of m and the elements of F vectors, NaN the lesser of any two.
template <typename T, int F>
__device__ __forceinline__ float largest(const uint4 (&x)[F], float m) {
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 top = __bfloat162bfloat162(__ushort_as_bfloat16(0xFF80));  // -inf
#pragma unroll
    for (int u = 0; u < F; ++u) {
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = __hmax2(top, reinterpret_cast<const __nv_bfloat162&>(w[i]));
    }
    return fmaxf(m, fmaxf(__low2float(top), __high2float(top)));
  } else {
#pragma unroll
    for (int u = 0; u < F; ++u)
      m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(x[u].x)), fmaxf(__uint_as_float(x[u].y), __uint_as_float(x[u].z))), __uint_as_float(x[u].w));
    return m;
  }
}

// A maximum and the sum of 2^(scale (x - maximum)) of the values behind it; a
// maximum of -inf is that of no values, or of nothing but -inf.
__device__ __forceinline__ float at_least(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float2 joined(float2 a, float2 b, float c) {
  const float m = fmaxf(a.x, b.x), n = at_least(m);
  return make_float2(m, __fmaf_rn(a.y, ex2((a.x - n) * c), b.y * ex2((b.x - n) * c)));
}

template <typename F>
__device__ __forceinline__ float2 warp_all(float2 v, F f) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = f(v, make_float2(__shfl_xor_sync(kAll, v.x, d), __shfl_xor_sync(kAll, v.y, d)));
  return v;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
  return x;
}

// A thread's picks of a token, HELD of them, THREADS apart: the teacher's logits, and
// where each stands in the range (kElsewhere, or kNone for no pick).
constexpr int64_t kElsewhere = -1, kNone = -2;
template <int THREADS, int HELD>
struct Picks {
  int64_t at[HELD];
  float t[HELD];

  __device__ __forceinline__ void load(const DistilArgs& a, uint64_t token) {
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const int k = threadIdx.x + j * THREADS;
      at[j] = -1;
      t[j] = -INFINITY;
      if (k >= a.picks) continue;
      const uint64_t i = token * a.picks + k;
      at[j] = a.wide_ids ? ((const int64_t*)a.ids)[i] : ((const int32_t*)a.ids)[i];
      t[j] = a.teacher_bf16 ? to_f32(((const bf16*)a.teacher)[i]) : ((const float*)a.teacher)[i];
    }
  }
  // Ids become places.  Apart from the loads, so that these are under way meanwhile.
  __device__ __forceinline__ void place(const DistilArgs& a) {
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const int64_t id = at[j];
      const bool pick = id >= 0 && id < a.vocabulary;
      if (!pick) t[j] = -INFINITY;
      at[j] = !pick ? kNone : id >= a.first && (uint64_t)(id - a.first) < a.width ? id - a.first : kElsewhere;
    }
  }
  __device__ __forceinline__ float best() const {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < HELD; ++j) m = fmaxf(m, t[j]);
    return m;
  }
  // exp of the teacher's logit against the best one, over the temperature
  __device__ __forceinline__ float weight(int j, float best, float tau) const {
    return at[j] == kNone ? 0.f : expf(__fdiv_rn(t[j] - at_least(best), tau));
  }
};

// The elements of a row [0, width) that a CTA of `split` takes: whole 16-byte
// vectors behind the `cut.head` elements before the first, split in equal parts;
// the elements beside the vectors are the first CTA's.
__device__ __forceinline__ uint64_t share(uint64_t nv, uint32_t rank, uint32_t split) { return nv * rank / split; }

// One token, by a cluster of CTAs that share its row; one pass, with the running
// maximum and sum in each thread.  The ids and the teacher's logits of the picks are
// fetched before the row, the student's behind it, when they are in the L2.
//
// Bound by DRAM: 4096 x 131072 bf16 in 150 us, 7.2 TB/s where the L2 holds a part from the
// call before; 8191 x 32768 in 81 us, 6.7 TB/s.  13.6 instructions an element bound it before
// (182 and 115 us); maxima of bf16 pairs and two values an instruction made them 8 (163
// and 98), and CTAs of 128 threads keep more rows under way.
template <typename T, int THREADS, int HELD>
__global__ void __launch_bounds__(THREADS) distil_kernel(const __grid_constant__ DistilArgs a, int split) {
  op_wait();
  constexpr int V = V16<T>, WARPS = THREADS / 32;
  __shared__ float2 of_warp[WARPS], of_cta[kMostCluster];
  __shared__ float best_of[WARPS];
  __shared__ float sum_of[3][WARPS];
  const uint64_t token = blockIdx.x / split;
  const uint32_t rank = blockIdx.x % split, tid = threadIdx.x;
  if (split > 1) cluster_arrive();  // that this CTA runs: others may write to its memory
  const T* row = (const T*)a.logits + token * a.ld;
  const float c = a.log2e_per_temperature;
  const Cut cut = cut_of<T, true>(row, a.width);
  const uint64_t v0 = share(cut.nv, rank, split), v1 = share(cut.nv, rank + 1, split);
  const T* body = row + cut.head;

  Picks<THREADS, HELD> picks;
  if (rank == 0) picks.load(a, token);
  float m = -INFINITY;
  F2 sum = f2(0.f);
  auto step = [&](auto number, uint64_t v) {
    constexpr int F = decltype(number)::value, P = V / 2;
    uint4 x[F];
#pragma unroll
    for (int u = 0; u < F; ++u) x[u] = ld16_if(body + (v + u * THREADS) * V, true);
#pragma unroll
    for (int u = 0; u < F; ++u) asm volatile("" : "+r"(x[u].x), "+r"(x[u].y), "+r"(x[u].z), "+r"(x[u].w));
    const float top = largest<T, F>(x, m), n = at_least(top);
    sum = sum * f2(ex2((m - n) * c));
    m = top;
#pragma unroll
    for (int u = 0; u < F; ++u) {
      F2 p[P];
      pairs_of<T>(x[u], p);
#pragma unroll
      for (int i = 0; i < P; ++i) sum = sum + ex2((p[i] + f2(-n)) * f2(c));
    }
  };
  uint64_t v = v0 + tid;
  for (; v + 3 * THREADS < v1; v += 4 * THREADS) step(std::integral_constant<int, 4>(), v);
  for (; v < v1; v += THREADS) step(std::integral_constant<int, 1>(), v);
  float s = both(sum);
  if (rank == 0 && tid < cut.beside) {
    const float x = to_f32(row[cut.at<V>(tid)]);
    s = __fmaf_rn(s, ex2((m - at_least(fmaxf(m, x))) * c), ex2((x - at_least(fmaxf(m, x))) * c));
    m = fmaxf(m, x);
  }
  float z[HELD];
  if (rank == 0) {
    picks.place(a);
#pragma unroll
    for (int j = 0; j < HELD; ++j) z[j] = picks.at[j] >= 0 ? to_f32(row[picks.at[j]]) : 0.f;
  }
  float2 ms = warp_all(make_float2(m, s), [c](float2 p, float2 q) { return joined(p, q, c); });
  float best = rank == 0 ? warp_max(picks.best()) : 0.f;
  if ((tid & 31) == 0) {
    of_warp[tid >> 5] = ms;
    best_of[tid >> 5] = best;
  }
  __syncthreads();
  ms = of_warp[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) ms = joined(ms, of_warp[w], c);
  if (split > 1) {
    cluster_wait();
    if (tid == 0) st_cluster(of_cta + rank, 0, ms);
    cluster_arrive();
    cluster_wait();
  }
  if (rank) return;
  if (split > 1) {
    ms = of_cta[0];
    for (int r = 1; r < split; ++r) ms = joined(ms, of_cta[r], c);
  }
  best = best_of[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) best = fmaxf(best, best_of[w]);

  // the sums over the picks: e, and of those in the range e (log-ratio) and e
  float all = 0.f, term = 0.f, mass = 0.f;
#pragma unroll
  for (int j = 0; j < HELD; ++j) {
    const float e = picks.weight(j, best, a.temperature);
    all += e;
    if (picks.at[j] < 0 || e == 0.f) continue;
    const float of_t = __fdiv_rn(picks.t[j] - at_least(best), a.temperature);
    const float of_z = __fdiv_rn(z[j] - at_least(ms.x), a.temperature);
    term = __fmaf_rn(e, of_t - of_z, term);
    mass += e;
  }
  all = warp_sum(all);
  term = warp_sum(term);
  mass = warp_sum(mass);
  if ((tid & 31) == 0) {
    sum_of[0][tid >> 5] = all;
    sum_of[1][tid >> 5] = term;
    sum_of[2][tid >> 5] = mass;
  }
  __syncthreads();
  if (tid) return;
  all = term = mass = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    all += sum_of[0][w];
    term += sum_of[1][w];
    mass += sum_of[2][w];
  }
  if (mass != 0.f) {  // NaN too
    term = __fdiv_rn(__fmaf_rn(-mass, logf(all), term), all);
    mass = __fdiv_rn(mass, all);
  }
  if (a.parts) {
    reinterpret_cast<Pack<float, 2>*>(a.parts)[2 * token] = {ms.x, ms.y};
    reinterpret_cast<Pack<float, 2>*>(a.parts)[2 * token + 1] = {term, mass};
  } else {
    a.loss[token] = mass == 0.f || ms.y == 0.f ? 0.f : a.scale * __fmaf_rn(mass, logf(ms.y), term);
    a.stats[2 * token] = ms.x;
    a.stats[2 * token + 1] = ms.y;
  }
}

// The parts of all ranges of a token, one thread for a token.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) distil_join_kernel(const __grid_constant__ DistilArgs a) {
  op_wait();
  const uint64_t token = (uint64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  if (token >= a.tokens) return;
  const float c = a.log2e_per_temperature;
  float2 ms = make_float2(-INFINITY, 0.f);
  for (int r = 0; r < a.ranks; ++r) {
    const float* p = a.parts + (r * a.tokens + token) * 4;
    ms = joined(ms, make_float2(p[0], p[1]), c);
  }
  float loss = 0.f, mass = 0.f;
  for (int r = 0; r < a.ranks; ++r) {
    const float* p = a.parts + (r * a.tokens + token) * 4;
    if (p[3] == 0.f) continue;
    mass += p[3];
    loss += __fmaf_rn(-p[3], __fdiv_rn(at_least(p[0]) - at_least(ms.x), a.temperature), p[2]);
  }
  a.loss[token] = mass == 0.f || ms.y == 0.f ? 0.f : a.scale * __fmaf_rn(mass, logf(ms.y), loss);
  a.stats[2 * token] = ms.x;
  a.stats[2 * token + 1] = ms.y;
}

// dz_j = G (Q p_j - the sum of q_k over the picks k of j), G = dL scale / temperature.
// The row is written without the picks first, then the picks' places again, by
// the CTA that wrote them, each by the first pick of its word.
//
// Bound by DRAM, reads and writes: 2047 x 65537 binary32 in 164 us, 6.5 TB/s; 4096 x 131072 bf16 in
// 316 us, 6.8.  Eight vectors in flight for each thread, evict-first stores and two
// vectors: level or slower (167, 173, 172 us of the former with 256 threads, four vectors
// 172).
template <typename T, bool SHIFT, int THREADS, int HELD>
__global__ void __launch_bounds__(THREADS) distil_grad_kernel(const __grid_constant__ DistilArgs a, int split) {
  op_wait();
  constexpr int V = V16<T>, WARPS = THREADS / 32;
  __shared__ float best_of[WARPS], sum_of[WARPS];
  __shared__ int64_t id_of[THREADS * HELD];
  __shared__ float q_of[THREADS * HELD];
  const uint64_t token = blockIdx.x / split;
  const uint32_t rank = blockIdx.x % split, tid = threadIdx.x;
  const T* row = (const T*)a.logits + token * a.ld;
  T* out = (T*)a.grad_logits + token * a.ldg;
  const float c = a.log2e_per_temperature;
  const Cut cut = cut_of<T, true>(out, a.width);
  const uint64_t v0 = share(cut.nv, rank, split), v1 = share(cut.nv, rank + 1, split);

  Picks<THREADS, HELD> picks;
  picks.load(a, token);
  const float of_max = a.stats[2 * token], total = a.stats[2 * token + 1], of_loss = a.grad_loss[token];
  picks.place(a);
  float z[HELD];
#pragma unroll
  for (int j = 0; j < HELD; ++j) z[j] = picks.at[j] >= 0 ? to_f32(row[picks.at[j]]) : 0.f;
  float best = warp_max(picks.best());
  if ((tid & 31) == 0) best_of[tid >> 5] = best;
  __syncthreads();
  best = best_of[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) best = fmaxf(best, best_of[w]);
  float e[HELD], all = 0.f;
#pragma unroll
  for (int j = 0; j < HELD; ++j) {
    all += e[j] = picks.weight(j, best, a.temperature);
    if (tid + j * THREADS < a.picks) {
      id_of[tid + j * THREADS] = picks.at[j];
      q_of[tid + j * THREADS] = e[j];
    }
  }
  all = warp_sum(all);
  if ((tid & 31) == 0) sum_of[tid >> 5] = all;
  __syncthreads();  // the picks' logits are read before any gradient is written in their place
  all = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) all += sum_of[w];
  const float m = at_least(of_max);
  const bool none = all == 0.f || total == 0.f;  // no picks, or nothing to take them from
  const float G = none ? 0.f : __fdiv_rn(of_loss * a.scale, a.temperature);
  const float f = none ? 0.f : __fdiv_rn(G, total) * __fdiv_rn(all, all);  // Q is 1, or NaN
  auto grad = [&](float z) { return none ? 0.f : f * ex2((z - m) * c); };

  const T* from = row + cut.head;
  T* to = out + cut.head;
  auto step = [&](auto number, uint64_t v) {
    constexpr int F = decltype(number)::value, P = V / 2;
    uint4 x[F];
#pragma unroll
    for (int u = 0; u < F; ++u) {
      const T* p = from + (v + u * THREADS) * V;
      if constexpr (SHIFT) {
        const Pack<T, V> r = ld_row_if<T, true>(p, true);
        memcpy(&x[u], &r, 16);
      } else {
        x[u] = ld16_if<Ld::kWritten>(p, true);
      }
    }
#pragma unroll
    for (int u = 0; u < F; ++u) asm volatile("" : "+r"(x[u].x), "+r"(x[u].y), "+r"(x[u].z), "+r"(x[u].w));
#pragma unroll
    for (int u = 0; u < F; ++u) {
      F2 p[P];
      pairs_of<T>(x[u], p);
#pragma unroll
      for (int i = 0; i < P; ++i) p[i] = none ? f2(0.f) : f2(f) * ex2((p[i] + f2(-m)) * f2(c));
      *reinterpret_cast<uint4*>(to + (v + u * THREADS) * V) = packed<T>(p);
    }
  };
  uint64_t v = v0 + tid;
  for (; v + 3 * THREADS < v1; v += 4 * THREADS) step(std::integral_constant<int, 4>(), v);
  for (; v < v1; v += THREADS) step(std::integral_constant<int, 1>(), v);
  if (rank == 0 && tid < cut.beside) {
    const uint64_t i = cut.at<V>(tid);
    out[i] = from_f32<T>(grad(to_f32(row[i])));
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < HELD; ++j) {
    const int k = tid + j * THREADS;
    if (k >= a.picks || picks.at[j] < 0 || none) continue;
    const uint64_t i = (uint64_t)picks.at[j];
    const bool beside = i < cut.head || i >= cut.head + cut.nv * V;
    const uint64_t v = (i - cut.head) / V;
    if (beside ? rank != 0 : v < v0 || v >= v1) continue;
    float q = e[j];
    bool first = true;
    for (int o = 0; o < a.picks; ++o)
      if (id_of[o] == picks.at[j] && o != k) {
        first = first && o > k;
        q += q_of[o];
      }
    if (first) out[i] = from_f32<T>(__fmaf_rn(-G, __fdiv_rn(q, all), grad(z[j])));
  }
}

// CTAs of a token: as many as bring the launch to `want`, in powers of two.
int split_of(uint64_t tokens, uint64_t width, uint64_t want) {
  int n = 1;
  while (n < kMostCluster && tokens * n * 2 <= want && width / (n * 2) >= 1024) n *= 2;
  return n;
}

// f(threads of a CTA, picks of a thread).  Fewer threads for a row mean that more
// rows are under way, of which each spends some time on its picks and sums: 8191 rows
// of 1000 / 8192 / 32768 bf16 words take 30 / 37 / 86 us with 256 threads each, 16 / 26 / 81 with
// 128, 12 / 24 / 82 with 64 (4096 x 131072: 156, 150, 154); the gradient 35 / 61 / 161, 17 / 45 / 162,
// 16 / 48 / 171 (2047 x 65537 binary32: 172, 187, 184, and 164 with 512).
struct RowSizes {
  uint64_t of64, of128;  // bytes of a row, at most
};
constexpr RowSizes kForward = {32 * 1024, UINT64_MAX}, kBackward = {8 * 1024, 64 * 1024};
template <typename F>
purlin_status with_threads(RowSizes most, uint64_t bytes, int picks, F f) {
  using std::integral_constant;
  if (bytes <= most.of64 && picks <= 64) return f(integral_constant<int, 64>(), integral_constant<int, 1>());
  if (bytes <= most.of128 && picks <= 128) return f(integral_constant<int, 128>(), integral_constant<int, 1>());
  return f(integral_constant<int, 512>(), integral_constant<int, PURLIN_MAX_PICKS / 512>());
}

}  // namespace

purlin_status launch_distil(const DistilArgs& a, int dtype, cudaStream_t s) {
  const int split = split_of(a.tokens, a.width, 4 * 152);
  return with_threads(kForward, a.width * (dtype == PL_F32 ? 4 : 2), a.picks, [&](auto threads, auto held) {
    constexpr int N = decltype(threads)::value, H = decltype(held)::value;
    if (dtype == PL_F32) return op_launch_cluster(split, distil_kernel<float, N, H>, a.tokens * split, N, 0, s, a, split);
    return op_launch_cluster(split, distil_kernel<bf16, N, H>, a.tokens * split, N, 0, s, a, split);
  });
}

purlin_status launch_distil_join(const DistilArgs& a, cudaStream_t s) {
  return op_launch(distil_join_kernel, (a.tokens + kJoinThreads - 1) / kJoinThreads, kJoinThreads, 0, s, a);
}

purlin_status launch_distil_grad(const DistilArgs& a, int dtype, cudaStream_t s) {
  const int split = split_of(a.tokens, a.width, 4 * 152);
  const uint64_t es = dtype == PL_F32 ? 4 : 2;
  // rows of both matrices at the same distance from a 16-byte boundary, all of them
  const bool even = (((uintptr_t)a.logits ^ (uintptr_t)a.grad_logits) & 15) == 0 && ((a.ld - a.ldg) * es & 15) == 0;
  return with_threads(kBackward, a.width * es, a.picks, [&](auto threads, auto held) {
    constexpr int N = decltype(threads)::value, H = decltype(held)::value;
    auto go = [&](auto fn) { return op_launch(fn, a.tokens * split, N, 0, s, a, split); };
    if (dtype == PL_F32) return even ? go(distil_grad_kernel<float, false, N, H>) : go(distil_grad_kernel<float, true, N, H>);
    return even ? go(distil_grad_kernel<bf16, false, N, H>) : go(distil_grad_kernel<bf16, true, N, H>);
  });
}

}  // namespace pl
