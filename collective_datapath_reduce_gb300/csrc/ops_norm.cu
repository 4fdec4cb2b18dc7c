// Layer norm of token rows behind a residual sum, and its gradient.
#include <type_traits>

#include "ops_common.cuh"

namespace pl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kMostThreads = 512;   // of a row
constexpr int kMostParts = 152;     // CTAs that leave sums of columns, at most
constexpr int kMostWidth = 8192;    // that a gradient's CTA holds in its registers

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}

// Sum over a row's threads, the same in each: a warp, or the whole CTA, whose
// `tmp` (a word for each warp) no earlier sum has used.
__device__ __forceinline__ float row_sum(float x, int tpr, float* tmp) {
  x = warp_sum(x);
  if (tpr == 32) return x;
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.f;
  for (int w = 0; w < tpr >> 5; ++w) x += tmp[w];
  return x;
}

// N elements from p; memory that this kernel may write in place, so not through
// the read-only path.
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> ld_in(const T* p, bool on) {
  if constexpr (N > 1) return ld_pack_if<T, N, Ld::kWritten>(p, on);
  Pack<T, N> r = zero_pack<T, N>();
  if (on) r.v[0] = *p;
  return r;
}

// N columns of a weight or bias, or `none` where there is no such vector.
template <typename W, int N>
__device__ __forceinline__ void ld_columns(const void* p, uint64_t c, bool on, float none, float (&out)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = none;
  if (!p || !on) return;
  const W* w = (const W*)p + c;
  constexpr int M = N * sizeof(W) > 16 ? 16 / sizeof(W) : N;
#pragma unroll
  for (int q = 0; q < N; q += M) {
    const Pack<W, M> r = *reinterpret_cast<const Pack<W, M>*>(w + q);
#pragma unroll
    for (int i = 0; i < M; ++i) out[q + i] = to_f32(r.v[i]);
  }
}

__device__ __forceinline__ float inverse(float variance, float eps) { return __frcp_rn(__fsqrt_rn(variance + eps)); }

// A row in the registers of tpr threads, NV vectors of N elements in each: the
// mean, then the squares of the distances from it, then the result.
template <typename T, typename W, int N, int NV>
__global__ void __launch_bounds__(kMostThreads) norm_kernel(const __grid_constant__ NormArgs a, int tpr) {
  op_wait();
  __shared__ float tmp[2][kMostThreads / 32];
  const int tid = threadIdx.x % tpr;
  const uint64_t row = (uint64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
  if (row >= a.tokens) return;
  const T* x = (const T*)a.x + row * a.ldx;
  Pack<T, N> p[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint64_t c = (uint64_t)(tid + j * tpr) * N;
    p[j] = ld_in<T, N>(x + c, c < a.width);
  }
  if (a.residual) {
    const T* r = (const T*)a.residual + row * a.ldr;
    Pack<T, N> q[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint64_t c = (uint64_t)(tid + j * tpr) * N;
      q[j] = ld_in<T, N>(r + c, c < a.width);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) p[j].v[i] = from_f32<T>(to_f32(p[j].v[i]) + to_f32(q[j].v[i]));
  }
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) s += to_f32(p[j].v[i]);
  const float mean = __fdiv_rn(row_sum(s, tpr, tmp[0]), (float)a.width);
  s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool on = (uint64_t)(tid + j * tpr) * N < a.width;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float d = to_f32(p[j].v[i]) - mean;
      if (on) s = __fmaf_rn(d, d, s);
    }
  }
  const float rstd = inverse(__fdiv_rn(row_sum(s, tpr, tmp[1]), (float)a.width), a.eps);
  if (a.stats && tid == 0) {
    a.stats[2 * row] = mean;
    a.stats[2 * row + 1] = rstd;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint64_t c = (uint64_t)(tid + j * tpr) * N;
    if (c >= a.width) break;
    if (a.total) st_pack((T*)a.total + row * a.ldt + c, p[j]);
    float w[N], b[N];
    ld_columns<W, N>(a.weight, c, true, 1.f, w);
    ld_columns<W, N>(a.bias, c, true, 0.f, b);
    Pack<T, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f32<T>(__fmaf_rn((to_f32(p[j].v[i]) - mean) * rstd, w[i], b[i]));
    st_pack((T*)a.y + row * a.ldy + c, o);
  }
}

// Rows of any width: read three times, twice of these from the caches.  Where y
// or the total lies on the input, a thread writes the elements that it reads.
template <typename T, typename W>
__global__ void __launch_bounds__(kMostThreads) norm_wide_kernel(const __grid_constant__ NormArgs a) {
  op_wait();
  __shared__ float tmp[2][kMostThreads / 32];
  const uint64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.ldx;
  const T* r = a.residual ? (const T*)a.residual + row * a.ldr : nullptr;
  auto value = [&](uint64_t c) {
    const float v = to_f32(x[c]);
    return r ? to_f32(from_f32<T>(v + to_f32(r[c]))) : v;
  };
  float s = 0.f;
  for (uint64_t c = threadIdx.x; c < a.width; c += kMostThreads) s += value(c);
  const float mean = __fdiv_rn(row_sum(s, kMostThreads, tmp[0]), (float)a.width);
  s = 0.f;
  for (uint64_t c = threadIdx.x; c < a.width; c += kMostThreads) {
    const float d = value(c) - mean;
    s = __fmaf_rn(d, d, s);
  }
  const float rstd = inverse(__fdiv_rn(row_sum(s, kMostThreads, tmp[1]), (float)a.width), a.eps);
  if (a.stats && threadIdx.x == 0) {
    a.stats[2 * row] = mean;
    a.stats[2 * row + 1] = rstd;
  }
  for (uint64_t c = threadIdx.x; c < a.width; c += kMostThreads) {
    const float v = value(c), w = a.weight ? to_f32(((const W*)a.weight)[c]) : 1.f;
    const float b = a.bias ? to_f32(((const W*)a.bias)[c]) : 0.f;
    if (a.total) ((T*)a.total)[row * a.ldt + c] = from_f32<T>(v);
    ((T*)a.y)[row * a.ldy + c] = from_f32<T>(__fmaf_rn((v - mean) * rstd, w, b));
  }
}

// ------------------------------------------------------------------ gradient
//
// With xh = (x - mean) / deviation and g = dy w:  dx = (g - mean(g) - xh mean(g
// xh)) / deviation (+ the gradient that reaches x beside the norm), and the
// columns' sums of dy xh and dy.  A CTA holds whole rows, its threads the
// columns' sums over the rows that pass through it; a second kernel adds the
// CTAs' sums, in order.

// Sums of two values over a row's threads: the tpr of a group, which has the
// CTA's barrier 1 + group and two rows of `tmp` that it uses in turn.
__device__ __forceinline__ float2 group_sum(float2 x, int tpr, int group, float2* tmp) {
  x.x = warp_sum(x.x);
  x.y = warp_sum(x.y);
  if (tpr == 32) return x;
  const int warp = (threadIdx.x >> 5) - group * (tpr >> 5);
  if ((threadIdx.x & 31) == 0) tmp[warp] = x;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
  x = make_float2(0.f, 0.f);
  for (int w = 0; w < tpr >> 5; ++w) {
    x.x += tmp[w].x;
    x.y += tmp[w].y;
  }
  return x;
}

template <typename T, typename W, int N, int NV>
__global__ void __launch_bounds__(kMostThreads) norm_grad_kernel(const __grid_constant__ NormArgs a, int tpr) {
  op_wait();
  extern __shared__ float sums[];  // [groups][2][width]
  __shared__ float2 tmp[2][kMostThreads / 32];
  const int tid = threadIdx.x % tpr, group = threadIdx.x / tpr, groups = blockDim.x / tpr;
  const uint32_t D = (uint32_t)a.width;
  const float per = __frcp_rn((float)D);
  float w[NV][N], dw[NV][N], db[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const uint32_t c = (uint32_t)(tid + j * tpr) * N;
    ld_columns<W, N>(a.weight, c, c < D, 1.f, w[j]);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[j][i] = db[j][i] = 0.f;
  }
  int turn = 0;
  for (uint64_t row = (uint64_t)blockIdx.x * groups + group; row < a.tokens; row += (uint64_t)gridDim.x * groups) {
    const T* x = (const T*)a.x + row * a.ldx;
    const T* dy = (const T*)a.grad_y + row * a.ldg;
    const T* dt = a.grad_total ? (const T*)a.grad_total + row * a.ldgt : nullptr;
    Pack<T, N> px[NV], pg[NV], pt[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t c = (uint32_t)(tid + j * tpr) * N;
      px[j] = ld_in<T, N>(x + c, c < D);
      pg[j] = ld_in<T, N>(dy + c, c < D);
      pt[j] = ld_in<T, N>(dt + c, dt && c < D);
    }
    const float mean = a.stats[2 * row], rstd = a.stats[2 * row + 1];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      // beside the row, dy is 0: no sum takes part of it
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = (to_f32(px[j].v[i]) - mean) * rstd, d = to_f32(pg[j].v[i]), g = d * w[j][i];
        dw[j][i] = __fmaf_rn(d, xh, dw[j][i]);
        db[j][i] += d;
        s.x += g;
        s.y = __fmaf_rn(g, xh, s.y);
      }
    }
    s = group_sum(s, tpr, group, tmp[turn] + group * (tpr >> 5));
    turn ^= 1;
    const float m = s.x * per, mx = s.y * per;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t c = (uint32_t)(tid + j * tpr) * N;
      if (c >= D) break;
      Pack<T, N> o;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = (to_f32(px[j].v[i]) - mean) * rstd, g = to_f32(pg[j].v[i]) * w[j][i];
        const float v = rstd * (__fmaf_rn(-xh, mx, g - m));
        o.v[i] = from_f32<T>(dt ? v + to_f32(pt[j].v[i]) : v);
      }
      st_pack((T*)a.y + row * a.ldy + c, o);
    }
  }
  if (!a.parts) return;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t c = (uint32_t)(tid + j * tpr) * N + i;
      if (c < D) {
        sums[(2 * group) * D + c] = dw[j][i];
        sums[(2 * group + 1) * D + c] = db[j][i];
      }
    }
  __syncthreads();
  for (uint32_t c = threadIdx.x; c < 2 * D; c += blockDim.x) {
    float v = 0.f;
    for (int g = 0; g < groups; ++g) v += sums[2 * g * D + c];
    a.parts[(uint64_t)blockIdx.x * 2 * D + c] = v;
  }
}

// The same for rows of any width, in two kernels: rows, and sums of columns.
template <typename T, typename W>
__global__ void __launch_bounds__(kMostThreads) norm_grad_wide_kernel(const __grid_constant__ NormArgs a) {
  op_wait();
  __shared__ float2 tmp[kMostThreads / 32];
  const uint64_t row = blockIdx.x;
  const T* x = (const T*)a.x + row * a.ldx;
  const T* dy = (const T*)a.grad_y + row * a.ldg;
  const float mean = a.stats[2 * row], rstd = a.stats[2 * row + 1], per = __frcp_rn((float)a.width);
  auto weight = [&](uint64_t c) { return a.weight ? to_f32(((const W*)a.weight)[c]) : 1.f; };
  float2 s = make_float2(0.f, 0.f);
  for (uint64_t c = threadIdx.x; c < a.width; c += kMostThreads) {
    const float xh = (to_f32(x[c]) - mean) * rstd, g = to_f32(dy[c]) * weight(c);
    s.x += g;
    s.y = __fmaf_rn(g, xh, s.y);
  }
  s = group_sum(s, kMostThreads, 0, tmp);
  const float m = s.x * per, mx = s.y * per;
  for (uint64_t c = threadIdx.x; c < a.width; c += kMostThreads) {
    const float xh = (to_f32(x[c]) - mean) * rstd, g = to_f32(dy[c]) * weight(c);
    float v = rstd * (__fmaf_rn(-xh, mx, g - m));
    if (a.grad_total) v += to_f32(((const T*)a.grad_total)[row * a.ldgt + c]);
    ((T*)a.y)[row * a.ldy + c] = from_f32<T>(v);
  }
}

constexpr int kColumns = 256;
template <typename T>
__global__ void __launch_bounds__(kColumns) norm_columns_kernel(const __grid_constant__ NormArgs a, int parts) {
  op_wait();
  const uint64_t part = blockIdx.x % parts, c = (uint64_t)(blockIdx.x / parts) * kColumns + threadIdx.x;
  if (c >= a.width) return;
  float dw = 0.f, db = 0.f;
#pragma unroll 4
  for (uint64_t row = part; row < a.tokens; row += parts) {
    const float d = to_f32(((const T*)a.grad_y)[row * a.ldg + c]);
    const float xh = (to_f32(((const T*)a.x)[row * a.ldx + c]) - a.stats[2 * row]) * a.stats[2 * row + 1];
    dw = __fmaf_rn(d, xh, dw);
    db += d;
  }
  a.parts[part * 2 * a.width + c] = dw;
  a.parts[(part * 2 + 1) * a.width + c] = db;
}

// The CTAs' sums of 32 columns, added in order by eight warps that share the CTAs.
template <typename W>
__global__ void __launch_bounds__(256) norm_join_kernel(const __grid_constant__ NormArgs a, int parts) {
  op_wait();
  __shared__ float tmp[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = blockIdx.x & 1;
  const uint64_t c = (uint64_t)(blockIdx.x >> 1) * 32 + lane;
  W* out = (W*)(which ? a.grad_bias : a.grad_weight);
  if (!out) return;
  float v = 0.f;
  if (c < a.width)
#pragma unroll 4
    for (int p = warp; p < parts; p += 8) v += a.parts[((uint64_t)p * 2 + which) * a.width + c];
  tmp[warp][lane] = v;
  __syncthreads();
  if (warp || c >= a.width) return;
  v = tmp[0][lane];
#pragma unroll
  for (int w = 1; w < 8; ++w) v += tmp[w][lane];
  out[c] = from_f32<W>(v);
}

bool even(const void* p, uint64_t ld, uint64_t size) { return !p || (((uintptr_t)p | ld * size) & 15u) == 0; }

int whole_warps(uint64_t threads) { return (int)((threads + 31) / 32 * 32); }

// f(vector's elements, vectors of a thread): the fewest with which 512 threads
// cover a row of up to kMostWidth elements.
template <int N, typename F>
purlin_status with_vectors(uint64_t width, F f) {
  using std::integral_constant;
  const uint64_t nv = (width + N - 1) / N;
  if (nv <= kMostThreads) return f(integral_constant<int, N>(), integral_constant<int, 1>());
  if (N == 8 || nv <= kMostThreads * 2) return f(integral_constant<int, N>(), integral_constant<int, 2>());
  if constexpr (N < 8) {
    if (N == 4 || nv <= kMostThreads * 4) return f(integral_constant<int, N>(), integral_constant<int, 4>());
    if constexpr (N < 4) return f(integral_constant<int, N>(), integral_constant<int, 16>());
  }
  return PL_ERR_UNSUPPORTED;
}

template <typename T, typename W>
purlin_status norm_t(const NormArgs& a, cudaStream_t s) {
  if (a.width > (uint64_t)kMostWidth) return op_launch(norm_wide_kernel<T, W>, a.tokens, kMostThreads, 0, s, a);
  constexpr int V = V16<T>;
  const uint64_t es = sizeof(T);
  const bool vec = a.width % V == 0 && even(a.x, a.ldx, es) && even(a.residual, a.ldr, es) && even(a.y, a.ldy, es) &&
                   even(a.total, a.ldt, es) && even(a.weight, 0, 1) && even(a.bias, 0, 1);
  auto go = [&](auto n, auto nv) {
    constexpr int N = decltype(n)::value, NV = decltype(nv)::value;
    const int tpr = whole_warps((a.width + N * NV - 1) / (N * NV)), per = tpr == 32 ? 4 : 1;
    return op_launch(norm_kernel<T, W, N, NV>, (a.tokens + per - 1) / per, tpr * per, 0, s, a, tpr);
  };
  return vec ? with_vectors<V>(a.width, go) : with_vectors<1>(a.width, go);
}

template <typename T, typename W>
purlin_status norm_grad_t(NormArgs a, cudaStream_t s) {
  constexpr int V = V16<T>;
  const uint64_t es = sizeof(T);
  const bool sums = a.grad_weight || a.grad_bias;
  if (!sums) a.parts = nullptr;
  int parts = 0;
  purlin_status st = PL_OK;
  if (a.width > (uint64_t)kMostWidth) {
    parts = (int)std::min<uint64_t>(kMostParts, a.tokens);
    // the columns first: dx may lie on what they read
    if (sums) st = op_launch(norm_columns_kernel<T>, (a.width + kColumns - 1) / kColumns * parts, kColumns, 0, s, a, parts);
    if (!st) st = op_launch(norm_grad_wide_kernel<T, W>, a.tokens, kMostThreads, 0, s, a);
  } else if (a.tokens) {
    const bool vec = a.width % V == 0 && even(a.x, a.ldx, es) && even(a.grad_y, a.ldg, es) && even(a.y, a.ldy, es) &&
                     even(a.grad_total, a.ldgt, es) && even(a.weight, 0, 1);
    auto go = [&](auto n, auto nv) {
      constexpr int N = decltype(n)::value, NV = decltype(nv)::value;
      const int tpr = whole_warps((a.width + N * NV - 1) / (N * NV)), groups = kMostThreads / tpr;
      parts = (int)std::min<uint64_t>(kMostParts, (a.tokens + groups - 1) / groups);
      const size_t smem = sums ? (size_t)groups * 2 * a.width * sizeof(float) : 0;
      const void* fn = (const void*)norm_grad_kernel<T, W, N, NV>;
      if (purlin_status e = op_smem(fn, smem, kMostThreads * N * NV * 2 * (int)sizeof(float))) return e;
      return op_launch(norm_grad_kernel<T, W, N, NV>, parts, tpr * groups, smem, s, a, tpr);
    };
    st = vec ? with_vectors<V>(a.width, go) : with_vectors<1>(a.width, go);
  }
  if (st || !sums) return st;
  return op_launch(norm_join_kernel<W>, (a.width + 31) / 32 * 2, 256, 0, s, a, parts);
}

}  // namespace

// Sums of a weight's and a bias's gradient for each of the CTAs that leave them.
size_t norm_grad_bytes(uint64_t tokens, uint64_t width) {
  return (size_t)(std::min<uint64_t>(kMostParts, tokens) * 2 * width * sizeof(float));
}

purlin_status launch_norm(const NormArgs& a, int dtype, int w_dtype, cudaStream_t s) {
  if (dtype == PL_F32) return w_dtype == PL_F32 ? norm_t<float, float>(a, s) : norm_t<float, bf16>(a, s);
  return w_dtype == PL_F32 ? norm_t<bf16, float>(a, s) : norm_t<bf16, bf16>(a, s);
}

purlin_status launch_norm_grad(const NormArgs& a, int dtype, int w_dtype, cudaStream_t s) {
  if (dtype == PL_F32) return w_dtype == PL_F32 ? norm_grad_t<float, float>(a, s) : norm_grad_t<float, bf16>(a, s);
  return w_dtype == PL_F32 ? norm_grad_t<bf16, float>(a, s) : norm_grad_t<bf16, bf16>(a, s);
}

}  // namespace pl
