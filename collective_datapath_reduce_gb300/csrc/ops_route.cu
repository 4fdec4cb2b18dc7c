// Routing of tokens to experts, and its gradient.
//
// One warp holds one token's logits, VPT neighbouring experts in each lane's
// registers, as keys: a binary32 value mapped to an unsigned integer of the
// same order (0 = the expert may not be picked), so that the best of the row
// is one integer max across the warp and ties fall to the lowest lane, which
// holds the lowest expert.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "ops_common.cuh"

namespace pl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 8;  // tokens per CTA

// Order-preserving map to unsigned; -inf and NaN map to 0, below everything.
// Adding +0 first makes -0 and +0 one key.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float of_key(uint32_t k) {
  return k == 0 ? -INFINITY : __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}

// Binary32 operations in the order of the formula, each rounded: the scores
// that decide between experts are the same as any other IEEE evaluation of it.
__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-x))); }

template <typename T, int VPT>
__device__ __forceinline__ void load_logits(const T* row, int lane, int experts, bool vec, float (&x)[VPT]) {
  const int e0 = lane * VPT;
  constexpr int N = VPT * sizeof(T) > 16 ? 16 / sizeof(T) : VPT;
  if (vec) {
    if (e0 < experts) {
#pragma unroll
      for (int q = 0; q < VPT; q += N) {
        const Pack<T, N> p = ld_pack<T, N>(row + e0 + q);
#pragma unroll
        for (int i = 0; i < N; ++i) x[q + i] = to_f32(p.v[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) x[i] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) x[i] = e0 + i < experts ? to_f32(row[e0 + i]) : -INFINITY;
  }
}

// Largest logit of the row, 0 where there is none; the sum of exp(x - best).
template <int VPT>
__device__ __forceinline__ void softmax_of(const float (&x)[VPT], int lane, int experts, float* best, float* sum) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) m = max(m, key_of(x[i]));
  m = __reduce_max_sync(kAll, m);
  *best = m ? of_key(m) : 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (lane * VPT + i < experts) s += expf(__fsub_rn(x[i], *best));
  *sum = warp_sum(s);
}

// Keeps the keys of the `kept` best groups.  `val` (shared, one warp's own):
// every expert's value of the group score; P lanes scan one group's.
template <int VPT>
__device__ __forceinline__ void keep_groups(uint32_t (&key)[VPT], const float* val, int lane, const RouteArgs& a) {
  const int n = a.experts / a.groups;
  int P = 32;
  while (P * a.groups > 32) P >>= 1;
  const int g = lane / P, q = lane % P;
  float one = -INFINITY, two = -INFINITY;
  if (g < a.groups) {
    for (int i = q; i < n; i += P) {
      const float v = val[g * n + i];
      two = fmaxf(two, fminf(one, v));
      one = fmaxf(one, v);
    }
  }
  for (int d = 1; d < P; d <<= 1) {
    const float o1 = __shfl_xor_sync(kAll, one, d), o2 = __shfl_xor_sync(kAll, two, d);
    two = fmaxf(fmaxf(two, o2), fminf(one, o1));
    one = fmaxf(one, o1);
  }
  const float of_group = a.best == 2 && two > -INFINITY ? __fadd_rn(one, two) : one;
  uint32_t gk = g < a.groups && q == 0 ? key_of(of_group) : 0;
  uint32_t keep = 0;  // bit g: group g
  for (int r = 0; r < a.kept; ++r) {
    const uint32_t top = __reduce_max_sync(kAll, gk);
    if (top == 0) break;
    const int who = __ffs(__ballot_sync(kAll, gk == top)) - 1;
    if (lane == who) gk = 0;
    keep |= 1u << (who / P);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = lane * VPT + i;
    if (e < a.experts && !(keep >> (e / n) & 1u)) key[i] = 0;
  }
}

template <typename T, int VPT>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteArgs a, int vec) {
  op_wait();
  extern __shared__ float shared[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t t = (uint64_t)blockIdx.x * kWarps + warp;
  if (t >= a.tokens) return;
  const T* row = (const T*)a.logits + t * a.ld;
  float x[VPT];
  load_logits<T, VPT>(row, lane, a.experts, vec, x);
  float best = 0.f, sum = 1.f;
  if (!a.sigmoid) softmax_of<VPT>(x, lane, a.experts, &best, &sum);

  uint32_t key[VPT];
  float* val = shared + warp * a.experts;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = lane * VPT + i;
    key[i] = key_of(x[i]);
    if (a.bias && key[i]) {
      const float s = a.sigmoid ? sigmoid(x[i]) : __fdiv_rn(expf(__fsub_rn(x[i], best)), sum);
      key[i] = key_of(__fadd_rn(s, a.bias[e]));
    }
    if (a.groups > 1 && e < a.experts) {
      float v = of_key(key[i]);
      if (a.best == 2 && !a.bias && key[i]) v = a.sigmoid ? sigmoid(x[i]) : expf(__fsub_rn(x[i], best));
      val[e] = v;
    }
  }
  if (a.groups > 1) {
    __syncwarp();
    keep_groups<VPT>(key, val, lane, a);
  }

  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) mine = max(mine, key[i]);
  int id = -1;  // lane j: pick j
  for (int j = 0; j < a.top_k; ++j) {
    const uint32_t top = __reduce_max_sync(kAll, mine);
    if (top == 0) break;
    const int who = __ffs(__ballot_sync(kAll, mine == top)) - 1;
    int e = 0;
    if (lane == who) {
      bool found = false;
      mine = 0;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (!found && key[i] == top) {
          found = true;
          e = lane * VPT + i;
          key[i] = 0;
        }
        mine = max(mine, key[i]);
      }
    }
    e = __shfl_sync(kAll, e, who);
    if (lane == j) id = e;
  }
  float w = 0.f;
  if (id >= 0) {
    const float v = to_f32(row[id]);
    w = a.sigmoid ? sigmoid(v) : __fdiv_rn(expf(__fsub_rn(v, best)), sum);
  }
  if (a.renormalise) w = __fdiv_rn(w, warp_sum(w) + 1e-20f);
  if (lane < a.top_k) {
    a.ids[t * a.top_k + lane] = id;
    a.weights[t * a.top_k + lane] = id >= 0 ? w * a.scale : 0.f;
  }
}

// With s the scores, S the sum of the picked ones (+ 1e-20) and dw the
// weights' gradient, ds_j = scale (dw_j - sum_l dw_l s_l / S) / S, or scale
// dw_j without renormalising.  Softmax: dx_i = s_i (ds_i - sum_j s_j ds_j);
// sigmoid: dx_i = ds_i s_i (1 - s_i).  The bias only chooses: no gradient.
template <typename T, int VPT>
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(const __grid_constant__ RouteArgs a, int vec) {
  op_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t t = (uint64_t)blockIdx.x * kWarps + warp;
  if (t >= a.tokens) return;
  const T* row = (const T*)a.logits + t * a.ld;
  int id = -1;
  float dw = 0.f;
  if (lane < a.top_k) {
    id = a.ids[t * a.top_k + lane];
    if (id < 0 || id >= a.experts) id = -1;
    else dw = a.grad_weights[t * a.top_k + lane] * a.scale;
  }
  float x[VPT], best = 0.f, sum = 1.f;
  if (!a.sigmoid) {
    load_logits<T, VPT>(row, lane, a.experts, vec, x);
    softmax_of<VPT>(x, lane, a.experts, &best, &sum);
  }
  float s = 0.f;
  if (id >= 0) {
    const float v = to_f32(row[id]);
    s = a.sigmoid ? sigmoid(v) : __fdiv_rn(expf(__fsub_rn(v, best)), sum);
  }
  float ds = dw;
  if (a.renormalise) {
    const float S = warp_sum(s) + 1e-20f;
    const float mean = __fdiv_rn(warp_sum(dw * s), S);
    ds = id >= 0 ? __fdiv_rn(dw - mean, S) : 0.f;
  }
  const bool any = __any_sync(kAll, id >= 0);
  float dot = 0.f, pick = ds;
  if (a.sigmoid) pick = ds * s * (1.f - s);
  else dot = warp_sum(ds * s);

  float g[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) g[i] = 0.f;
  for (int j = 0; j < a.top_k; ++j) {
    const int e = __shfl_sync(kAll, id, j);
    const float v = __shfl_sync(kAll, pick, j);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (e == lane * VPT + i) g[i] += v;
  }
  T* out = (T*)a.grad_logits + t * a.grad_ld;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = lane * VPT + i;
    if (!a.sigmoid) g[i] = any ? __fdiv_rn(expf(__fsub_rn(x[i], best)), sum) * (g[i] - dot) : 0.f;
    if (e < a.experts) out[e] = from_f32<T>(g[i]);
  }
}

// Experts per lane: the smallest power of two that covers them with 32 lanes.
template <typename F>
purlin_status with_vpt(int experts, F f) {
  if (experts <= 32) return f(std::integral_constant<int, 1>());
  if (experts <= 64) return f(std::integral_constant<int, 2>());
  if (experts <= 128) return f(std::integral_constant<int, 4>());
  if (experts <= 256) return f(std::integral_constant<int, 8>());
  if (experts <= 512) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

template <typename T, int VPT>
int vec_ok(const RouteArgs& a) {
  const int need = std::min<int>(16, VPT * (int)sizeof(T));
  return a.experts % VPT == 0 && vec_bytes((uint64_t)(uintptr_t)a.logits | a.ld * sizeof(T)) >= need;
}

}  // namespace

purlin_status launch_route(const RouteArgs& a, int dtype, cudaStream_t s) {
  const uint64_t grid = (a.tokens + kWarps - 1) / kWarps;
  const size_t smem = a.groups > 1 ? (size_t)kWarps * a.experts * sizeof(float) : 0;  // at most 32 KiB
  return with_vpt(a.experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (dtype == PL_F32) return op_launch(route_kernel<float, V>, grid, kWarps * 32, smem, s, a, vec_ok<float, V>(a));
    return op_launch(route_kernel<bf16, V>, grid, kWarps * 32, smem, s, a, vec_ok<bf16, V>(a));
  });
}

purlin_status launch_route_grad(const RouteArgs& a, int dtype, cudaStream_t s) {
  const uint64_t grid = (a.tokens + kWarps - 1) / kWarps;
  return with_vpt(a.experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (dtype == PL_F32) return op_launch(route_grad_kernel<float, V>, grid, kWarps * 32, 0, s, a, vec_ok<float, V>(a));
    return op_launch(route_grad_kernel<bf16, V>, grid, kWarps * 32, 0, s, a, vec_ok<bf16, V>(a));
  });
}

}  // namespace pl
