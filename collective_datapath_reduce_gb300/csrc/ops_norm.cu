// Layer norm of token rows behind a residual sum.
#include "ops_norm.cuh"

namespace pl {
namespace {

__device__ __forceinline__ float inverse(float variance, float eps) { return __frcp_rn(__fsqrt_rn(variance + eps)); }

// Rows pass through a CTA's registers, NV vectors in each of a row's threads, and
// its weights stay there.  A warp takes the mean of its part and the squares of the
// distances from that; the warps' means and squares join to the row's, (sum of
// squares) + n (mean of the part - mean)^2 each, behind one barrier.
//
// 16384 x 5120 bf16 with a residual: 99 us, 6.8 TB/s, the copy bandwidth.  A CTA for each
// row, weights read anew and two barriers, took 150 us; rows by the ring and weights
// kept 136; two values an instruction 107, and fewer instructions for addresses the
// rest.  1024 threads with 8 elements each: 136 us.  Rows of odd width go element by element: 1.8
// to 2.4 times the time that their bytes take (3001 x 1537 binary32: 10.6 us, 16000 x 4095 bf16: 94),
// bound by the instructions of an element.  Vectors cut at the rows' ends instead made the
// warps with the ends the slowest (115 us) and all others wait.
template <typename T, typename W, Lie LIE, int NV>
__global__ void __launch_bounds__(kMostThreads) norm_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ Ring ring) {
  op_wait();
  extern __shared__ __align__(16) char smem[];
  __shared__ float2 tmp[2][kMostThreads / 32];
  using Rows = Stream<T, LIE, NV, 2>;
  constexpr int P = Rows::P, N = Rows::N;
  Rows in(ring, smem, a.width);
  const int tid = in.tid, tpr = in.tpr, warps = tpr >> 5, warp = tid >> 5, lane = threadIdx.x & 31;
  const uint64_t rows = (uint64_t)gridDim.x * ring.groups;
  uint64_t row = (uint64_t)blockIdx.x * ring.groups + in.group;
  in.take(row, rows, a.tokens);
  const bool second = a.residual != nullptr;
  in.open(0, a.x, a.ldx, row, rows);
  if (second) in.open(1, a.residual, a.ldr, row, rows);
  in.begin();
  F2 w[P], b[P];
  in.template columns<W>(a.weight, 1.f, w);
  in.template columns<W>(a.bias, 0.f, b);
  // elements of a warp (of a row of a few lanes: all)
  auto part = [&](int of) {
    if (warps < 2) return in.width;
    int n = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (of * 32 + j * tpr) * N;
      n += max(0, min(in.width - c, 32 * N));
    }
    return n;
  };
  const float mine = (float)part(warp), per_mine = mine > 0.f ? __frcp_rn(mine) : 0.f, per = __frcp_rn((float)in.width);
  // lane i joins warp i's
  const float of_lane = lane < warps ? (float)part(lane) : 0.f, per_lane = of_lane > 0.f ? __frcp_rn(of_lane) : 0.f;
  int turn = 0;
  T* y = in.place(a.y, a.ldy, row);
  T* total = a.total ? in.place(a.total, a.ldt, row) : nullptr;
  // the rows of a warp's lanes need not end together
  for (; __any_sync(kAll, row < a.tokens); row += rows) {
    const uint32_t at = in.next();
    F2 v[P], sum = f2(0.f);
    in.get(at, 0, (const T*)a.x + row * a.ldx, v);
    if (second) {
      F2 q[P];
      in.get(at, 1, (const T*)a.residual + row * a.ldr, q);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        v[i] = v[i] + q[i];
        if constexpr (sizeof(T) == 2) v[i] = pair_of(bf16x2_of(v[i]));  // the norm is of what is stored
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) sum = LIE != Lie::kWhole ? fma2(in.times(i), v[i], sum) : sum + v[i];
    float s = lanes_sum(both(sum), tpr), mean = s * per_mine;
    sum = f2(0.f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const F2 d = v[i] + f2(-mean);
      sum = fma2(LIE != Lie::kWhole ? in.times(i) * d : d, d, sum);
    }
    float squares = lanes_sum(both(sum), tpr);
    if (warps > 1) {
      float2* t = tmp[turn] + in.group * warps;
      turn ^= 1;
      if (lane == 0) t[warp] = make_float2(s, squares);
      group_barrier(in.group, tpr);
      const float2 of = lane < warps ? t[lane] : make_float2(0.f, 0.f);
      mean = warp_sum(of.x) * per;
      const float off = __fmaf_rn(of.x, per_lane, -mean);
      squares = warp_sum(__fmaf_rn(of_lane * off, off, of.y));
    }
    const float rstd = inverse(squares * per, a.eps);
    if (row >= a.tokens) continue;
    if (a.stats && tid == 0) {
      a.stats[2 * row] = mean;
      a.stats[2 * row + 1] = rstd;
    }
    if (total) {
      in.put(total, v);
      total += rows * a.ldt;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = fma2((v[i] + f2(-mean)) * f2(rstd), w[i], b[i]);
    in.put(y, v);
    y += rows * a.ldy;
  }
}

// Sum over a CTA, the same in each thread; `tmp`: a word for each warp, which no earlier sum has used.
__device__ __forceinline__ float cta_sum(float x, float* tmp) {
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.f;
  for (int w = 0; w < kMostThreads / 32; ++w) x += tmp[w];
  return x;
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
  const float mean = __fdiv_rn(cta_sum(s, tmp[0]), (float)a.width);
  s = 0.f;
  for (uint64_t c = threadIdx.x; c < a.width; c += kMostThreads) {
    const float d = value(c) - mean;
    s = __fmaf_rn(d, d, s);
  }
  const float rstd = inverse(__fdiv_rn(cta_sum(s, tmp[1]), (float)a.width), a.eps);
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

template <typename T, typename W>
purlin_status norm_t(const NormArgs& a, cudaStream_t s) {
  constexpr uint64_t es = sizeof(T);
  const bool aligned = a.width % V16<T> == 0 && even(a.x, a.ldx, es) && even(a.residual, a.ldr, es) && even(a.y, a.ldy, es) &&
                       even(a.total, a.ldt, es);
  auto go = [&](auto lie, auto nv, int tpr) {
    constexpr Lie L = decltype(lie)::value;
    constexpr int NV = decltype(nv)::value;
    const Ring r = ring_of<T>(L, a.width, tpr, a.residual ? 2 : 1);
    const uint64_t grid = std::min<uint64_t>(kSms, (a.tokens + r.groups - 1) / r.groups);
    if (purlin_status e = op_smem((const void*)norm_kernel<T, W, L, NV>, r.smem(), kSmem)) return e;
    return op_launch(norm_kernel<T, W, L, NV>, grid, tpr * r.groups, r.smem(), s, a, r);
  };
  return with_shape<T>(aligned, a.width, go, [&] { return op_launch(norm_wide_kernel<T, W>, a.tokens, kMostThreads, 0, s, a); });
}

}  // namespace

purlin_status launch_norm(const NormArgs& a, int dtype, int w_dtype, cudaStream_t s) {
  if (dtype == PL_F32) return w_dtype == PL_F32 ? norm_t<float, float>(a, s) : norm_t<float, bf16>(a, s);
  return w_dtype == PL_F32 ? norm_t<bf16, float>(a, s) : norm_t<bf16, bf16>(a, s);
}

}  // namespace pl
