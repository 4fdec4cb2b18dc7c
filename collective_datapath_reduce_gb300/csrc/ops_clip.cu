// The global norm of many tensors, and their scaled, clipped copies.
//
// The first kernel leaves each CTA's sum of squares; the second adds them in a
// fixed order in every CTA (so all agree, and from call to call), derives the
// factor and writes.  Squares are added in binary32 over a few vectors of one
// thread and from there on in binary64.
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

// Calls vec(first element) for the 16-byte vectors and one(element) for the
// others of elements [e0, e1) at p; `q` shares p's alignment or vec is not used.
template <typename T, typename V, typename O>
__device__ __forceinline__ void walk(const T* p, bool aligned, uint64_t e0, uint64_t e1, V vec, O one) {
  constexpr int N = 16 / sizeof(T);
  if (!aligned) {
    for (uint64_t i = e0 + threadIdx.x; i < e1; i += kThreads) one(i);
    return;
  }
  const uint64_t off = ((uintptr_t)(p + e0) & 15) / sizeof(T);
  const uint64_t v0 = min(e1, off ? e0 + N - off : e0);
  const uint64_t v1 = v0 + (e1 - v0) / N * N;
  for (uint64_t i = v0 + (uint64_t)threadIdx.x * N; i < v1; i += (uint64_t)kThreads * N) vec(i);
  if (threadIdx.x < N && e0 + threadIdx.x < v0) one(e0 + threadIdx.x);
  if (threadIdx.x < N && v1 + threadIdx.x < e1) one(v1 + threadIdx.x);
}

__device__ __forceinline__ double block_sum(double s, double* tmp) {
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x / 32] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += tmp[w];
  return s;
}

template <typename T, int M>
__global__ void __launch_bounds__(kThreads) squares_kernel(const __grid_constant__ Table<M> a) {
  op_wait();
  __shared__ double tmp[kThreads / 32];
  constexpr int N = 16 / sizeof(T);
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < a.first[a.n]; c += gridDim.x) {
    const int t = tensor_of(a, c);
    const uint64_t e0 = (uint64_t)(c - a.first[t]) * kChunk, e1 = min(a.t[t].n, e0 + kChunk);
    const T* p = (const T*)a.t[t].in;
    float s = 0.f;
    walk<T>(
        p, true, e0, e1,
        [&](uint64_t i) {
          const Pack<T, N> x = ld_pack<T, N>(p + i);
#pragma unroll
          for (int k = 0; k < N; ++k) s = __fmaf_rn(to_f32(x.v[k]), to_f32(x.v[k]), s);
        },
        [&](uint64_t i) { s = __fmaf_rn(to_f32(p[i]), to_f32(p[i]), s); });
    sum += (double)s;
  }
  sum = block_sum(sum, tmp);
  if (threadIdx.x == 0) a.parts[a.part0 + blockIdx.x] = sum;
}

// norm and factor, by every CTA alike
template <int M>
__device__ __forceinline__ float factor_of(const Table<M>& a, double* tmp, bool tell) {
  double s = 0.0;
  for (int i = threadIdx.x; i < a.nparts; i += kThreads) s += a.parts[i];
  const float norm = (float)(sqrt(block_sum(s, tmp)) * fabs((double)a.scale));
  if (tell && threadIdx.x == 0) *a.norm = norm;
  if (isinf(a.max_norm)) return a.scale;
  const float f = __fdiv_rn(a.max_norm, norm + 1e-6f);
  return (f < 1.f || isnan(f) ? f : 1.f) * a.scale;
}

template <typename T, int M>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table<M> a) {
  op_wait();
  __shared__ double tmp[kThreads / 32];
  constexpr int N = 16 / sizeof(T);
  const float f = factor_of(a, tmp, a.part0 == 0 && blockIdx.x == 0);
  for (uint32_t c = blockIdx.x; c < a.first[a.n]; c += gridDim.x) {
    const int t = tensor_of(a, c);
    const uint64_t e0 = (uint64_t)(c - a.first[t]) * kChunk, e1 = min(a.t[t].n, e0 + kChunk);
    const T* p = (const T*)a.t[t].in;
    T* o = (T*)a.t[t].out;
    walk<T>(
        p, (((uintptr_t)p ^ (uintptr_t)o) & 15) == 0, e0, e1,
        [&](uint64_t i) {
          Pack<T, N> x = *reinterpret_cast<const Pack<T, N>*>(p + i);
#pragma unroll
          for (int k = 0; k < N; ++k) x.v[k] = from_f32<T>(to_f32(x.v[k]) * f);
          st_pack<T, N>(o + i, x);
        },
        [&](uint64_t i) { o[i] = from_f32<T>(to_f32(p[i]) * f); });
  }
}

template <int M>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Table<M> a) {
  op_wait();
  __shared__ double tmp[kThreads / 32];
  factor_of(a, tmp, true);
}

uint64_t chunks_of(uint64_t n) { return (n + kChunk - 1) / kChunk; }

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
  auto fill = [&](size_t l) {
    a.n = (int)std::min<size_t>(M, n - l * M);
    uint64_t c = 0;
    for (int i = 0; i < a.n; ++i) {
      a.t[i] = t[l * M + i];
      a.first[i] = (uint32_t)c;
      c += chunks_of(a.t[i].n);  // far below 2^32 for any memory
    }
    a.first[a.n] = (uint32_t)c;
    return c;
  };
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
