// Routing of tokens to experts, and its gradient.
//
// One warp holds one token's logits, VPT neighbouring experts in each lane's
// registers.  The best of the row is one maximum across the warp, and ties fall
// to the lowest lane, which holds the lowest expert.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "ops_common.cuh"

namespace pl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 4;  // tokens per CTA (2, 4, 8, 16: 17.3, 17.5, 17.9, 19.1 us for the case at route_kernel)

// Largest value of the warp, in every lane.
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// A key that can be compared: NaN, the lesser of every maximum, becomes -inf,
// which may not be picked.
__device__ __forceinline__ float key_of(float x) { return fmaxf(x, -INFINITY); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}

// Binary32 operations in the order of the formula, each rounded: the scores
// that decide between experts are the same as any other IEEE evaluation of it.
__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(__fadd_rn(1.f, expf(-x))); }

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
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPT; ++i) m = fmaxf(m, x[i]);
  m = warp_max(m);
  *best = m > -INFINITY ? m : 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (lane * VPT + i < experts) s += expf(__fsub_rn(x[i], *best));
  *sum = warp_sum(s);
}

// The better two of two pairs.
__device__ __forceinline__ void merge_two(float& one, float& two, float o1, float o2) {
  two = fmaxf(fmaxf(two, o2), fminf(one, o1));
  one = fmaxf(one, o1);
}

__device__ __forceinline__ uint32_t lowest(uint32_t bits) { return bits & (0u - bits); }

// Bits of the first lanes of the `kept` best groups.  2^shift neighbouring
// lanes hold a group's best two values (first group in lane 0).
__device__ __forceinline__ uint32_t kept_groups(float one, float two, int shift, int lane, const RouteArgs& a) {
  for (int d = 1; d < 1 << shift; d <<= 1) {
    const float o1 = __shfl_xor_sync(kAll, one, d), o2 = __shfl_xor_sync(kAll, two, d);
    merge_two(one, two, o1, o2);
  }
  const float value = a.best == 2 && two > -INFINITY ? __fadd_rn(one, two) : one;
  const bool first = (lane & ((1 << shift) - 1)) == 0 && lane >> shift < a.groups;
  float key = first ? key_of(value) : -INFINITY;
  uint32_t keep = 0;
  for (int r = 0; r < a.kept; ++r) {
    const float top = warp_max(key);
    if (!(top > -INFINITY)) break;
    const uint32_t best = lowest(__ballot_sync(kAll, key == top));
    if (best == 1u << lane) key = -INFINITY;
    keep |= best;
  }
  return keep;
}

// A lane's best two keys and their experts, equal ones in order.
struct Two {
  float k1, k2;
  int e1, e2;
};
template <int VPT>
__device__ __forceinline__ Two best_two(const float (&key)[VPT], int e0) {
  Two t = {-INFINITY, -INFINITY, 0, 0};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const bool first = key[i] > t.k1, second = key[i] > t.k2;
    t.k2 = first ? t.k1 : fmaxf(t.k2, key[i]);
    t.e2 = first ? t.e1 : second ? e0 + i : t.e2;
    t.k1 = fmaxf(t.k1, key[i]);
    t.e1 = first ? e0 + i : t.e1;
  }
  return t;
}

// The picks are taken one by one: each lane offers its best key left, one
// maximum across the warp finds the best of the row.  A lane keeps its best
// two keys ready and searches its registers again only after its second pick.
//
// Bound by the instructions of a row (860), not by its bytes (17 MB, 2.6
// us).  16384 tokens, 256 experts, 8 picks, sigmoid, bias, 4 of 8 groups by their
// best two: 35 us with a search at every pick, 22 us with two keys ready, 19 us
// with shifts for the divisions by a group's lanes and the pick passed through
// shared memory by the lane that offers it (a bit scan takes 4 cycles per SM, a
// maximum or a ballot 1), 17.5 us with keys compared as they are, not mapped to
// integers, and the bias read in vectors.  Of that a pick takes 0.6 us, the
// sigmoids 3 us, the groups 3 us.
template <typename T, int VPT>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteArgs a, int vec) {
  op_wait();
  extern __shared__ float shared[];
  __shared__ int picks[kWarps][PURLIN_MAX_TOP_K];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * VPT;
  const uint64_t t = (uint64_t)blockIdx.x * kWarps + warp;
  if (t >= a.tokens) return;
  const T* row = (const T*)a.logits + t * a.ld;
  float x[VPT];
  load_logits<T, VPT>(row, lane, a.experts, vec & 1, x);
  float best = 0.f, sum = 1.f;
  if (!a.sigmoid) softmax_of<VPT>(x, lane, a.experts, &best, &sum);

  float key[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) key[i] = key_of(x[i]);
  if (a.bias && e0 < a.experts) {
    float bias[VPT];
    if (vec & 2) {
      constexpr int N = VPT < 4 ? VPT : 4;
#pragma unroll
      for (int q = 0; q < VPT; q += N) {
        const Pack<float, N> p = *reinterpret_cast<const Pack<float, N>*>(a.bias + e0 + q);
#pragma unroll
        for (int i = 0; i < N; ++i) bias[q + i] = p.v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) bias[i] = e0 + i < a.experts ? __ldg(a.bias + e0 + i) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const float s = a.sigmoid ? sigmoid(x[i]) : __fdiv_rn(expf(__fsub_rn(x[i], best)), sum);
      key[i] = key[i] > -INFINITY ? key_of(__fadd_rn(s, bias[i])) : -INFINITY;
    }
  }
  // what counts for a group of the expert with this key: s + bias or the
  // logit, or, of a sum of two without a bias, s (softmax: times the sum, and
  // +inf for a logit of +inf, whose s is none)
  const bool by_score = a.best == 2 && !a.bias;
  auto value = [&](float k) {
    if (!by_score || !(k > -INFINITY)) return k;
    return a.sigmoid ? sigmoid(k) : k == INFINITY ? k : expf(__fsub_rn(k, best));
  };

  if (a.groups > 1 && a.group_shift < 0) {
    // groups that cut through lanes: through shared memory, 2^shift lanes scan a group
    float* val = shared + warp * a.experts;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (e0 + i < a.experts) val[e0 + i] = value(key[i]);
    __syncwarp();
    const int n = a.group_size;
    int shift = 5;
    while (a.groups << shift > 32) --shift;
    float one = -INFINITY, two = -INFINITY;
    if (lane >> shift < a.groups)
      for (int i = lane & ((1 << shift) - 1); i < n; i += 1 << shift) merge_two(one, two, val[(lane >> shift) * n + i], -INFINITY);
    const uint32_t keep = kept_groups(one, two, shift, lane, a);
    int g = e0 / n, left = n - e0 % n;  // the group of expert e0 + i, and its experts from there on
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (!(keep >> (g << shift & 31) & 1u)) key[i] = -INFINITY;
      if (--left == 0) {
        ++g;
        left = n;
      }
    }
  }
  Two b = best_two<VPT>(key, e0);
  if (a.groups > 1 && a.group_shift >= 0) {
    const uint32_t keep = kept_groups(value(b.k1), value(b.k2), a.group_shift, lane, a);
    if (!(keep >> (lane & -1 << a.group_shift) & 1u)) b.k1 = -INFINITY;
  }

  int* pick = picks[warp];
  int j = 0, last_e = 0;
  float last = 0.f;    // this lane's last pick
  bool ready = true;   // b.k2 is the best key behind b.k1
  bool look = false;   // b.k1 is not known, and +inf until it is looked for
  while (j < a.top_k) {
    const float top = warp_max(b.k1);
    if (fabsf(top) == INFINITY) {
      if (top < 0.f) break;
      if (__any_sync(kAll, look)) {
        if (look) {  // the best key behind the lane's last pick
          look = false;
          b.k1 = -INFINITY;
#pragma unroll
          for (int i = 0; i < VPT; ++i) {
            const bool behind = key[i] < last || (key[i] == last && e0 + i > last_e);
            if (behind && key[i] > b.k1) {
              b.k1 = key[i];
              b.e1 = e0 + i;
            }
          }
        }
        continue;
      }
    }
    if (lowest(__ballot_sync(kAll, b.k1 == top)) == 1u << lane) {
      pick[j] = last_e = b.e1;
      last = b.k1;
      look = !ready;
      b.k1 = ready ? b.k2 : INFINITY;
      b.e1 = b.e2;
      ready = false;
    }
    ++j;
  }
  __syncwarp();
  const int id = lane < j ? pick[lane] : -1;
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
// sigmoid: dx_i = ds_i s_i (1 - s_i).  The bias only chooses: no gradient.  One
// warp per token as in the forward pass; the picks' parts are added to the lanes
// that hold their experts.  At 8191 x 60 bf16, 4 picks, 5 us: 2 MB in all, so two
// round trips and the launch.
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
    load_logits<T, VPT>(row, lane, a.experts, vec & 1, x);
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

// 2^shift lanes hold a group of n experts, or -1 where a group's end cuts a lane.
int shift_of(int n, int vpt) {
  if (n % vpt) return -1;
  for (int s = 0; s <= 5; ++s)
    if (n / vpt == 1 << s) return s;
  return -1;
}

template <typename T, int VPT>
int vec_ok(const RouteArgs& a) {
  const uint64_t need = std::min<uint64_t>(16, VPT * sizeof(T));
  const bool whole = a.experts % VPT == 0;  // every lane's experts exist or none
  const int logits = whole && ((uint64_t)(uintptr_t)a.logits | a.ld * sizeof(T)) % need == 0;
  const int bias = whole && (uintptr_t)a.bias % std::min<uint64_t>(16, VPT * sizeof(float)) == 0;
  return logits | bias << 1;
}

}  // namespace

purlin_status launch_route(const RouteArgs& in, int dtype, cudaStream_t s) {
  const uint64_t grid = (in.tokens + kWarps - 1) / kWarps;
  return with_vpt(in.experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    RouteArgs a = in;
    a.group_size = a.experts / a.groups;
    a.group_shift = shift_of(a.group_size, V);
    // the groups' values, at most 16 KiB
    const size_t smem = a.groups > 1 && a.group_shift < 0 ? (size_t)kWarps * a.experts * sizeof(float) : 0;
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
