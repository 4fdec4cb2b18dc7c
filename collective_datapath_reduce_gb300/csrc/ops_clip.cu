// The global norm of many tensors, and their scaled, clipped copies.
//
// The first kernel leaves each CTA's sum of squares; the second adds them in a
// fixed order in every CTA (so all agree, and from call to call), derives the
// factor and writes.  Few elements go through one CTA of one kernel.  Squares
// are added in binary32 over a few vectors of one thread and from there on in
// binary64.
//
// Past the L2 the values have to be read twice and written once: 238 M binary32
// values in 180 tensors take 138 + 290 us, 6.9 and 6.6 TB/s.  In the first
// kernel shares in one piece for each CTA beat strided ones (163 us) because a
// share looks its tensor up once; in the second they were slower (300 us).  Its
// stores are evict-first: 428 us in all against 430 with ordinary ones, in place
// 434 against 426.
#include <math.h>

#include <type_traits>

#include "ops_common.cuh"

namespace pl {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxParts = 2048;    // CTAs' partial sums, at most
constexpr uint64_t kChunk = 16384;  // elements of one piece of work

// The tensors of one launch travel in the kernel's parameters.
constexpr int kFew = 64, kMany = 1024;
template <int M>
struct Table {
  ClipTensor t[M];
  uint32_t first[M + 1];  // first chunk of each tensor
  int n;
  double* parts;       // all CTAs' sums, of all launches
  int part0, nparts;   // this launch's first; their number over all launches
  float scale, max_norm;
  float* norm;
};

template <int M>
__device__ __forceinline__ int tensor_of(const Table<M>& a, uint32_t chunk) {
  int lo = 0, hi = a.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// CTA b's pieces are share(b) .. share(b + 1): neighbours, so that the tensor
// is looked up once and then followed.
__device__ __forceinline__ uint32_t share(uint32_t chunks, uint32_t b) {
  return (uint32_t)((uint64_t)chunks * b / gridDim.x);
}

// Runs vec(vector, first element, whether there is one) for the 16-byte vectors
// of elements [e0, e1) at p, F of a thread in flight at a time, and one(element)
// for the elements beside them.
template <int THREADS, int F, Ld HOW, typename T, typename V, typename O>
__device__ __forceinline__ void walk(const T* p, bool aligned, uint64_t e0, uint64_t e1, V vec, O one) {
  constexpr int N = 16 / sizeof(T);
  const uint32_t tid = threadIdx.x % THREADS;
  if (!aligned) {
    for (uint64_t i = e0 + tid; i < e1; i += THREADS) one(i);
    return;
  }
  const uint64_t off = ((uintptr_t)(p + e0) & 15) / sizeof(T);
  const uint64_t v0 = min(e1, off ? e0 + N - off : e0);
  const uint32_t nv = (uint32_t)((e1 - v0) / N);
  for (uint32_t v = tid; v < nv; v += THREADS * F) {
    Pack<T, N> x[F];
#pragma unroll
    for (int u = 0; u < F; ++u) x[u] = ld_pack_if<T, N, HOW>(p + v0 + (uint64_t)(v + u * THREADS) * N, v + u * THREADS < nv);
#pragma unroll
    for (int u = 0; u < F; ++u) pin(x[u]);
#pragma unroll
    for (int u = 0; u < F; ++u) vec(x[u], v0 + (uint64_t)(v + u * THREADS) * N, v + u * THREADS < nv);
  }
  const uint64_t v1 = v0 + (uint64_t)nv * N;
  if (tid < N && e0 + tid < v0) one(e0 + tid);
  if (tid < N && v1 + tid < e1) one(v1 + tid);
}

// Squares of elements [e0, e1) at p, this thread's part: in binary32, or, where
// they do not fit (or are not numbers), once more in binary64.  HOW: kWritten
// where the same kernel writes in place later.
template <int THREADS, int F, Ld HOW, typename T>
__device__ __forceinline__ double squares(const T* p, uint64_t e0, uint64_t e1) {
  float s = 0.f;
  walk<THREADS, F, HOW, T>(
      p, true, e0, e1,
      [&](const auto& x, uint64_t, bool) {  // zeros where there is none
#pragma unroll
        for (int k = 0; k < 16 / (int)sizeof(T); ++k) s = __fmaf_rn(to_f32(x.v[k]), to_f32(x.v[k]), s);
      },
      [&](uint64_t i) { s = __fmaf_rn(to_f32(p[i]), to_f32(p[i]), s); });
  if (s <= 1e38f) return (double)s;
  double w = 0.0;
  walk<THREADS, 1, HOW, T>(
      p, true, e0, e1,
      [&](const auto& x, uint64_t, bool) {
        for (int k = 0; k < 16 / (int)sizeof(T); ++k) w += (double)to_f32(x.v[k]) * (double)to_f32(x.v[k]);
      },
      [&](uint64_t i) { w += (double)to_f32(p[i]) * (double)to_f32(p[i]); });
  return w;
}

// In place, an element is loaded and stored by the same thread, and by no other.
template <int THREADS, int F, typename T>
__device__ __forceinline__ void scale(const T* p, T* o, uint64_t e0, uint64_t e1, float f) {
  walk<THREADS, F, Ld::kWritten, T>(
      p, (((uintptr_t)p ^ (uintptr_t)o) & 15) == 0, e0, e1,
      [&](auto& x, uint64_t i, bool on) {
#pragma unroll
        for (int k = 0; k < 16 / (int)sizeof(T); ++k) x.v[k] = from_f32<T>(to_f32(x.v[k]) * f);
        if (on) st_pack_once(o + i, x);
      },
      [&](uint64_t i) { o[i] = from_f32<T>(to_f32(p[i]) * f); });
}

// Sum over the CTA, the same in every thread.  Binary64 additions are slow
// here, so they are few in a row: by lanes, then by warps.
template <int THREADS>
__device__ __forceinline__ double block_sum(double s, double* tmp) {
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x / 32] = s;
  __syncthreads();
  constexpr int W = THREADS / 32;
  s = tmp[threadIdx.x % W];
#pragma unroll
  for (int d = W / 2; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  return s;
}

// Apart, so that it is a call that is not made and no work whose result is not taken.
__device__ __noinline__ float wide_norm(double sum, float size) { return (float)(sqrt(sum) * (double)size); }

// The factor, given the sum of squares; one thread writes the norm.
template <int M>
__device__ __forceinline__ float factor_of(const Table<M>& a, double sum, bool tell) {
  // binary64 square roots take long: only where the sum is outside binary32,
  // and then the scale too is applied before the rounding, which it may decide
  const float size = fabsf(a.scale), norm = sum > 1e-30 && sum < 1e38 ? __fsqrt_rn((float)sum) * size : wide_norm(sum, size);
  if (tell) *a.norm = norm;
  if (isinf(a.max_norm)) return a.scale;
  const float f = __fdiv_rn(a.max_norm, norm + 1e-6f);
  return (f < 1.f || isnan(f) ? f : 1.f) * a.scale;
}

template <int M>
__device__ __forceinline__ double sum_of_parts(const Table<M>& a, double* tmp) {
  double s = 0.0;
  for (int i = threadIdx.x; i < a.nparts; i += kThreads) s += a.parts[i];
  return block_sum<kThreads>(s, tmp);
}

template <typename T, int M>
__global__ void __launch_bounds__(kThreads, 2) squares_kernel(const __grid_constant__ Table<M> a) {
  op_wait();
  __shared__ double tmp[kThreads / 32];
  double sum = 0.0;
  const uint32_t chunks = a.first[a.n];
  const uint32_t c0 = share(chunks, blockIdx.x), c1 = share(chunks, blockIdx.x + 1);
  int t = tensor_of(a, c0);
  for (uint32_t c = c0; c < c1; ++c) {
    while (c >= a.first[t + 1]) ++t;
    const uint64_t e0 = (uint64_t)(c - a.first[t]) * kChunk;
    sum += squares<kThreads, 8, Ld::kOnce>((const T*)a.t[t].in, e0, min(a.t[t].n, e0 + kChunk));
  }
  sum = block_sum<kThreads>(sum, tmp);
  if (threadIdx.x == 0) a.parts[a.part0 + blockIdx.x] = sum;
}

template <typename T, int M>
__global__ void __launch_bounds__(kThreads, 2) scale_kernel(const __grid_constant__ Table<M> a) {
  op_wait();
  __shared__ double tmp[kThreads / 32];
  const float f = factor_of(a, sum_of_parts(a, tmp), a.part0 == 0 && blockIdx.x == 0 && threadIdx.x == 0);
  const uint32_t chunks = a.first[a.n];
  for (uint32_t d = blockIdx.x; d < chunks; d += gridDim.x) {
    // The end first: the SMs hold half of squares_kernel's CTAs at once, so the
    // second half of the list was read last, and some of it is still in the L2
    // (from the start 433 against 428 us; 26 M values 54 against 53).
    const uint32_t c = chunks - 1 - d;
    const int t = tensor_of(a, c);
    const uint64_t e0 = (uint64_t)(c - a.first[t]) * kChunk;
    scale<kThreads, 8>((const T*)a.t[t].in, (T*)a.t[t].out, e0, min(a.t[t].n, e0 + kChunk), f);
  }
}

template <int M>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Table<M> a) {
  op_wait();
  __shared__ double tmp[kThreads / 32];
  factor_of(a, sum_of_parts(a, tmp), threadIdx.x == 0);
}

// Few elements: one CTA, a warp for each piece of kSmallChunk elements.  On the
// device the two kernels are level (20000 values: 8.8 and 8.4 us) and later ahead
// (60000: 13.7 and 8.4), but the second launch costs the host 2.5 us, and few
// elements wait for the host.
constexpr int kSmallThreads = 1024;
constexpr uint64_t kSmallChunk = 1024, kSmallMost = 32 * 1024;
template <typename T>
__global__ void __launch_bounds__(kSmallThreads) clip_small_kernel(const __grid_constant__ Table<kFew> a, int write) {
  op_wait();
  __shared__ double tmp[kSmallThreads / 32];
  constexpr int F = kSmallChunk * sizeof(T) / (32 * 16);  // a piece in one go
  const uint32_t chunks = a.first[a.n], warp = threadIdx.x / 32;
  double sum = 0.0;
  for (uint32_t c = warp; c < chunks; c += kSmallThreads / 32) {
    const int t = tensor_of(a, c);
    const uint64_t e0 = (uint64_t)(c - a.first[t]) * kSmallChunk;
    sum += squares<32, F, Ld::kWritten>((const T*)a.t[t].in, e0, min(a.t[t].n, e0 + kSmallChunk));
  }
  sum = block_sum<kSmallThreads>(sum, tmp);
  const float f = factor_of(a, sum, threadIdx.x == 0);
  for (uint32_t c = warp; write && c < chunks; c += kSmallThreads / 32) {
    const int t = tensor_of(a, c);
    const uint64_t e0 = (uint64_t)(c - a.first[t]) * kSmallChunk;
    scale<32, F>((const T*)a.t[t].in, (T*)a.t[t].out, e0, min(a.t[t].n, e0 + kSmallChunk), f);
  }
}

template <typename T, int M>
purlin_status clip_t(const ClipTensor* t, size_t n, float scale, float max_norm, bool write, float* norm, double* partials,
                     int sm_count, cudaStream_t s) {
  // a launch takes M tensors at most; with more launches than partial sums
  // allow for full grids, the grids shrink
  const size_t launches = std::max<size_t>(1, (n + M - 1) / M);
  if (launches > (size_t)kMaxParts) return PL_ERR_UNSUPPORTED;
  const int most = std::max<int>(1, std::min<int>(sm_count * 4, kMaxParts / (int)launches));
  Table<M> a = {};
  a.parts = partials;
  a.scale = scale;
  a.max_norm = max_norm;
  a.norm = norm;
  uint64_t elements = 0;
  for (size_t i = 0; i < n; ++i) elements += t[i].n;
  const bool small = M == kFew && elements <= kSmallMost;
  const uint64_t piece = small ? kSmallChunk : kChunk;
  auto fill = [&](size_t l) {
    a.n = (int)std::min<size_t>(M, n - l * M);
    uint64_t c = 0;
    for (int i = 0; i < a.n; ++i) {
      a.t[i] = t[l * M + i];
      a.first[i] = (uint32_t)c;
      c += (a.t[i].n + piece - 1) / piece;  // far below 2^32 for any memory
    }
    a.first[a.n] = (uint32_t)c;
    return c;
  };
  if constexpr (M == kFew)
    if (small) {
      fill(0);
      return op_launch(clip_small_kernel<T>, 1, kSmallThreads, 0, s, a, (int)write);
    }
  int parts = 0;
  for (size_t l = 0; l < launches; ++l) {
    const uint64_t c = fill(l);
    a.part0 = parts;
    const int grid = (int)std::min<uint64_t>(c, most);
    if (purlin_status st = op_launch(squares_kernel<T, M>, grid, kThreads, 0, s, a)) return st;
    parts += grid;
  }
  a.nparts = parts;
  if (!write || n == 0) return op_launch(norm_kernel<M>, 1, kThreads, 0, s, a);
  for (size_t l = 0; l < launches; ++l) {
    const uint64_t c = fill(l);
    a.part0 = (int)l;  // launch 0 writes the norm
    if (purlin_status st = op_launch(scale_kernel<T, M>, std::min<uint64_t>(c, most), kThreads, 0, s, a)) return st;
  }
  return PL_OK;
}

}  // namespace

size_t clip_bytes() { return kMaxParts * sizeof(double); }

purlin_status launch_clip(const ClipTensor* t, size_t n, int dtype, float scale, float max_norm, bool write, float* norm,
                          double* partials, int sm_count, cudaStream_t s) {
  auto go = [&](auto m) {
    constexpr int M = decltype(m)::value;
    return dtype == PL_F32 ? clip_t<float, M>(t, n, scale, max_norm, write, norm, partials, sm_count, s)
                           : clip_t<bf16, M>(t, n, scale, max_norm, write, norm, partials, sm_count, s);
  };
  return n <= kFew ? go(std::integral_constant<int, kFew>()) : go(std::integral_constant<int, kMany>());
}

}  // namespace pl
