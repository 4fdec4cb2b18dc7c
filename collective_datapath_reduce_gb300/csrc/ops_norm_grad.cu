// The layer norm's gradient.
//
// With xh = (x - mean) / deviation and g = dy w:  dx = (g - mean(g) - xh mean(g
// xh)) / deviation (+ the gradient that reaches x beside the norm), and the
// columns' sums of dy xh and dy.  A CTA holds whole rows, its threads the
// columns' sums over the rows that pass through it; a second kernel adds the
// CTAs' sums, in order, or, of few rows, the CTAs of one cluster do.
//
// 8192 x 4096 bf16 with the residual's gradient: 50 us, 46 of them before the join; 5.4 TB/s, 80%
// of the copy bandwidth (39.5 us).  What is left is beside the rows: two launches, the
// ring's start and the sums' way out (200 rows take 9.1 us).  Loads when a row needs them:
// 112 us; by the ring 60; two values an instruction 54; sums across a warp by its
// halves and one round of loads in the join 50.  Launching the join early cost 2 us (its CTAs
// take the places of this kernel's last ones), and so did launching it at this one's
// end; CTAs of 768 threads at 80 registers took 64 us, of 1024 with 8 elements each 89.
// With 24 bf16 values a thread (kPart, 3) the registers are at their limit and some are
// spilled: 8192 x 5120 in 74 us, half the copy bandwidth (37.1 us).
#include "ops_norm.cuh"

namespace pl {
namespace {

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of the shared memory of the cluster's CTA `rank`, where p is in this one's.
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
  uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// Sums of two values over a row's threads; `tmp`: two words for each warp, of two
// rows that are used in turn.  The halves of a warp take one value each.
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int d = 8; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
__device__ __forceinline__ float2 group_sum(float2 x, int tpr, int group, float* tmp) {
  if (tpr < 32) return make_float2(lanes_sum(x.x, tpr), lanes_sum(x.y, tpr));
  const int lane = threadIdx.x & 31, half = lane >> 4, warps = tpr >> 5;
  const float other = __shfl_xor_sync(kAll, half ? x.x : x.y, 16);
  float v = half_sum((half ? x.y : x.x) + other);
  if (warps > 1) {
    if ((lane & 15) == 0) tmp[2 * ((threadIdx.x >> 5) - group * warps) + half] = v;
    group_barrier(group, tpr);
    v = half_sum((lane & 15) < warps ? tmp[2 * (lane & 15) + half] : 0.f);
  }
  return make_float2(__shfl_sync(kAll, v, 0), __shfl_sync(kAll, v, 16));
}

template <typename T, typename W, Lie LIE, int NV>
__global__ void __launch_bounds__(kMostThreads) norm_grad_kernel(const __grid_constant__ NormArgs a,
                                                                 const __grid_constant__ Ring ring, int alone) {
  op_wait();
  extern __shared__ __align__(16) char smem[];  // the ring, then [groups][2][width] sums
  __shared__ float tmp[2][kMostThreads / 16];
  using Rows = Stream<T, LIE, NV, 3>;
  constexpr int P = Rows::P, N = Rows::N;
  Rows in(ring, smem, a.width);
  const int tpr = in.tpr, group = in.group, groups = ring.groups, D = in.width;
  const uint64_t rows = (uint64_t)gridDim.x * groups;
  // groups of one number take neighbouring rows, so that the last rows, fewer than
  // groups, fall on all CTAs (20011 x 520 binary32: 25.5 us, 26.0 with neighbours to a
  // CTA; in the forward pass that is the better way, 102 us and 105)
  uint64_t row = (uint64_t)group * gridDim.x + blockIdx.x;
  in.take(row, rows, a.tokens);
  const bool third = a.grad_total != nullptr;
  in.open(0, a.x, a.ldx, row, rows);
  in.open(1, a.grad_y, a.ldg, row, rows);
  if (third) in.open(2, a.grad_total, a.ldgt, row, rows);
  in.begin();
  const float per = __frcp_rn((float)D);
  F2 w[P], dw[P], db[P];
  in.template columns<W>(a.weight, 1.f, w);
#pragma unroll
  for (int i = 0; i < P; ++i) dw[i] = db[i] = f2(0.f);
  int turn = 0;
  T* dx = in.place(a.y, a.ldy, row);
  float2 ahead = row < a.tokens ? make_float2(a.stats[2 * row], a.stats[2 * row + 1]) : make_float2(0.f, 0.f);
  // the rows of a warp's lanes need not end together
  for (; __any_sync(kAll, row < a.tokens); row += rows) {
    const uint32_t at = in.next();
    const bool live = row < a.tokens;
    const float mean = ahead.x, rstd = ahead.y;
    if (row + rows < a.tokens) ahead = make_float2(a.stats[2 * (row + rows)], a.stats[2 * (row + rows) + 1]);
    const T *of_x = (const T*)a.x + row * a.ldx, *of_g = (const T*)a.grad_y + row * a.ldg;
    F2 x[P], g[P], sum = f2(0.f), sum_xh = f2(0.f);
    if (live) {
      in.get(at, 0, of_x, x);
      in.get(at, 1, of_g, g);
      // beside the row the weights are 0, and the columns' sums nobody's
#pragma unroll
      for (int i = 0; i < P; ++i) {
        x[i] = (x[i] + f2(-mean)) * f2(rstd);
        dw[i] = fma2(g[i], x[i], dw[i]);
        db[i] = db[i] + g[i];
        g[i] = g[i] * w[i];
        sum = sum + g[i];
        sum_xh = fma2(g[i], x[i], sum_xh);
      }
    }
    float2 s = make_float2(both(sum), both(sum_xh));
    s = group_sum(s, tpr, group, tmp[turn] + group * (tpr >> 4));
    turn ^= 1;
    if (!live) continue;
    const F2 m = f2(-s.x * per), mx = f2(-s.y * per);
    if constexpr (P > 8) {  // too many registers to hold them while the warps wait
      in.get(at, 0, of_x, x);
      in.get(at, 1, of_g, g);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        x[i] = (x[i] + f2(-mean)) * f2(rstd);
        g[i] = g[i] * w[i];
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = f2(rstd) * fma2(x[i], mx, g[i] + m);
    if (third) {
      in.get(at, 2, (const T*)a.grad_total + row * a.ldgt, g);
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = x[i] + g[i];
    }
    in.put(dx, x);
    dx += rows * a.ldy;
  }
  if (!a.parts) return;
  copies_left<0>();
  __syncthreads();
  float *of_w = (float*)smem + 2 * group * D, *of_b = of_w + D;
#pragma unroll
  for (int i = 0; i < 2 * P; ++i) {
    const float2 vw = split(dw[i / 2]), vb = split(db[i / 2]);
    if (!in.there(i / N)) continue;
    of_w[in.column(i / N) + i % N] = i % 2 ? vw.y : vw.x;
    of_b[in.column(i / N) + i % N] = i % 2 ? vb.y : vb.x;
  }
  __syncthreads();
  float* sums = (float*)smem;
  for (int c = threadIdx.x; c < 2 * D; c += blockDim.x) {
    float v = 0.f;
    for (int g = 0; g < groups; ++g) v += sums[2 * g * D + c];
    if (alone) sums[c] = v;
    else a.parts[(uint64_t)blockIdx.x * 2 * D + c] = v;
  }
  if (!alone) return;
  // the CTAs are one cluster, and take the columns in turn
  cluster_sync();
  for (int c = blockIdx.x * blockDim.x + threadIdx.x; c < 2 * D; c += gridDim.x * blockDim.x) {
    W* out = (W*)(c < D ? a.grad_weight : a.grad_bias);
    if (!out) continue;
    float v = 0.f;
    for (uint32_t r = 0; r < gridDim.x; ++r) v += ld_cluster(sums + c, r);
    out[c < D ? c : c - D] = from_f32<W>(v);
  }
  cluster_sync();  // before a CTA ends whose memory is read
}

// The same for rows of any width, in two kernels: rows, and sums of columns.
template <typename T, typename W>
__global__ void __launch_bounds__(kMostThreads) norm_grad_wide_kernel(const __grid_constant__ NormArgs a) {
  op_wait();
  __shared__ float tmp[kMostThreads / 16];
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

// The CTAs' sums of 32 columns, added in order by eight warps that share the CTAs,
// a warp's loads all at once.
constexpr int kJoinWarps = 8, kJoinLoads = (kSms + kJoinWarps - 1) / kJoinWarps;
template <typename W>
__global__ void __launch_bounds__(kJoinWarps * 32) norm_join_kernel(const __grid_constant__ NormArgs a, int parts) {
  op_wait();
  __shared__ float tmp[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = blockIdx.x & 1;  // the weight's or the bias's
  const uint64_t c = (uint64_t)(blockIdx.x >> 1) * 32 + lane;
  W* out = (W*)(which ? a.grad_bias : a.grad_weight);
  if (!out) return;
  float x[kJoinLoads], v = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinLoads; ++i) {
    const int p = warp + i * kJoinWarps;
    x[i] = ld1_if(a.parts + ((uint64_t)p * 2 + which) * a.width + c, p < parts && c < a.width);
  }
#pragma unroll
  for (int i = 0; i < kJoinLoads; ++i) v += x[i];
  tmp[warp][lane] = v;
  __syncthreads();
  if (warp || c >= a.width) return;
  v = tmp[0][lane];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) v += tmp[w][lane];
  out[c] = from_f32<W>(v);
}

// Few rows go through one cluster and one launch, kFewRows for each of its groups:
// the second launch costs the host 2 to 3 us (calls of 30 / 60 / 120 x 4096 bf16: 13.1 / 13.4 / 17.3 us in
// one, 15.8 / 15.5 / 15.8 in two; on the device 10.4 / 12.8 / 17.3 and 8.7 / 8.9 / 8.9).
constexpr int kCluster = 8, kFewRows = 4;

template <typename T, typename W>
purlin_status norm_grad_t(NormArgs a, cudaStream_t s) {
  constexpr uint64_t es = sizeof(T);
  const bool sums = a.grad_weight || a.grad_bias;
  if (!sums) a.parts = nullptr;
  int parts = 0;
  bool done = !sums;  // nothing is left to be joined
  const bool aligned = a.width % V16<T> == 0 && even(a.x, a.ldx, es) && even(a.grad_y, a.ldg, es) && even(a.y, a.ldy, es) &&
                       even(a.grad_total, a.ldgt, es);
  auto go = [&](auto lie, auto nv, int tpr) {
    constexpr Lie L = decltype(lie)::value;
    constexpr int NV = decltype(nv)::value;
    const Ring r = ring_of<T>(L, a.width, tpr, a.grad_total ? 3 : 2);
    const uint64_t rounds = (a.tokens + r.groups - 1) / r.groups;  // of one CTA
    const bool alone = rounds <= kCluster * kFewRows;
    parts = (int)std::min<uint64_t>(alone ? kCluster : kSms, rounds);
    if (alone)
      while (parts & (parts - 1)) ++parts;  // a power of two
    done = done || alone;
    const uint32_t of_sums = sums ? (uint32_t)(r.groups * 2 * a.width * sizeof(float)) : 0, smem = std::max(r.smem(), of_sums);
    if (purlin_status e = op_smem((const void*)norm_grad_kernel<T, W, L, NV>, smem, kSmem)) return e;
    return op_launch_cluster(alone ? parts : 1, norm_grad_kernel<T, W, L, NV>, parts, tpr * r.groups, smem, s, a, r, (int)alone);
  };
  auto wide = [&] {
    parts = (int)std::min<uint64_t>(kSms, a.tokens);
    // the columns first: dx may lie on what they read
    if (sums) {
      const uint64_t grid = (a.width + kColumns - 1) / kColumns * parts;
      if (purlin_status e = op_launch(norm_columns_kernel<T>, grid, kColumns, 0, s, a, parts)) return e;
    }
    return op_launch(norm_grad_wide_kernel<T, W>, a.tokens, kMostThreads, 0, s, a);
  };
  const purlin_status st = a.tokens ? with_shape<T>(aligned, a.width, go, wide) : PL_OK;
  if (st || done) return st;
  return op_launch(norm_join_kernel<W>, (a.width + 31) / 32 * 2, kJoinWarps * 32, 0, s, a, parts);
}

}  // namespace

// Sums of a weight's and a bias's gradient for each of the CTAs that leave them.
size_t norm_grad_bytes(uint64_t tokens, uint64_t width) {
  return (size_t)(std::min<uint64_t>(kSms, tokens) * 2 * width * sizeof(float));
}

purlin_status launch_norm_grad(const NormArgs& a, int dtype, int w_dtype, cudaStream_t s) {
  if (dtype == PL_F32) return w_dtype == PL_F32 ? norm_grad_t<float, float>(a, s) : norm_grad_t<float, bf16>(a, s);
  return w_dtype == PL_F32 ? norm_grad_t<bf16, float>(a, s) : norm_grad_t<bf16, bf16>(a, s);
}

}  // namespace pl
