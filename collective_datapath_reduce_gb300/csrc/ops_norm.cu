// Layer norm of token rows behind a residual sum, and its gradient.
#include <type_traits>

#include "ops_common.cuh"

namespace pl {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kMostThreads = 512;
constexpr int kSms = 152;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}

__device__ __forceinline__ void group_barrier(int group, int tpr) {
  if (tpr <= 32) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
}

// 16 bytes from global into shared memory, when they come.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_left() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
  return u;
}
template <typename T>
__device__ __forceinline__ float ld_shared1(uint32_t at) {
  if constexpr (sizeof(T) == 4) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
  } else {
    unsigned short x;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
    return __uint_as_float((uint32_t)x << 16);
  }
}

// How rows lie.  On 16-byte boundaries, and the threads' vectors fill them (kWhole)
// or reach past their ends, whole vectors (kPart); or any other way, element by
// element (kSingle).
enum class Lie { kWhole, kPart, kSingle };

// Rows on their way into shared memory.  A CTA is `groups` groups of tpr
// threads, a row each at a time; a group has `stages` slots, a row of each of n
// matrices in every one, so that stages - 1 rows are under way while one is
// worked on.  A thread copies the vectors that it uses, and waits for nobody
// else; kSingle's threads share the aligned granules that hold the row's bytes.
struct Ring {
  int n, stages, tpr, groups;
  uint32_t granules;  // of a row's slot
  uint32_t smem() const { return (uint32_t)(n * stages * groups) * granules * 16; }
};

// A thread's view of a row: NV vectors of N elements, tpr vectors apart, as P
// pairs.  For a vector beside the row it reads the row's first and counts it 0 times.
template <typename T, Lie LIE, int NV, int M>
struct Stream {
  static constexpr bool SINGLE = LIE == Lie::kSingle;
  static constexpr int N = SINGLE ? 1 : V16<T>, P = N * NV / 2, S = N * (int)sizeof(T);  // S: bytes of a vector
  const char* from[M];   // the next row to fetch, of each matrix; but for kSingle: this thread's first vector
  uint64_t step[M];      // bytes to the one behind it
  uint64_t left;         // rows to fetch
  uint32_t bytes;        // of a row
  uint32_t matrix, stage, slots, in, out, first;  // of shared memory, in bytes
  int tid, group, tpr, stages, width, n;  // n: matrices

  __device__ __forceinline__ Stream(const Ring& r, const void* smem, uint64_t columns) {
    tpr = r.tpr;
    stages = r.stages;
    n = r.n;
    tid = threadIdx.x % tpr;
    group = threadIdx.x / tpr;
    width = (int)columns;
    bytes = (uint32_t)width * sizeof(T);
    matrix = (uint32_t)r.groups * r.granules * 16;
    stage = matrix * n;
    slots = stage * stages;
    in = out = 0;
    first = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)group * r.granules * 16;
  }
  // Rows `row`, row + rows, .. of `tokens`.
  __device__ __forceinline__ void take(uint64_t row, uint64_t rows, uint64_t tokens) {
    left = row < tokens ? (tokens - row - 1) / rows + 1 : 0;
  }
  __device__ __forceinline__ void open(int m, const void* p, uint64_t ld, uint64_t row, uint64_t rows) {
    from[m] = (const char*)p + row * ld * sizeof(T) + (SINGLE ? 0 : tid * 16);
    step[m] = rows * ld * sizeof(T);
  }
  // This thread's first vector of a row of a matrix that is written.
  __device__ __forceinline__ T* place(void* p, uint64_t ld, uint64_t row) const {
    return (T*)p + row * ld + tid * N;
  }
  // Bytes from the row's start to vector j, its column, and whether it is there.
  __device__ __forceinline__ uint32_t offset(int j) const { return (uint32_t)(tid + j * tpr) * S; }
  __device__ __forceinline__ int column(int j) const { return (tid + j * tpr) * N; }
  __device__ __forceinline__ bool there(int j) const { return LIE == Lie::kWhole || offset(j) < bytes; }
  // How often a pair counts.
  __device__ __forceinline__ F2 times(int pair) const {
    if constexpr (SINGLE) return f2(there(2 * pair) ? 1.f : 0.f, there(2 * pair + 1) ? 1.f : 0.f);
    return f2(there(pair * 2 / N) ? 1.f : 0.f);
  }

  // One more row, or an empty step behind the last.
  __device__ __forceinline__ void fetch() {
    if (left) {
      --left;
#pragma unroll
      for (int m = 0; m < M; ++m) {
        if (m >= n) break;
        const uint32_t to = first + in + m * matrix;
        if constexpr (SINGLE) {
          const uint32_t off = (uint32_t)((uintptr_t)from[m] & 15u), last = off + bytes;
          for (uint32_t i = tid * 16; i < last; i += tpr * 16) copy16(to + i, from[m] - off + i);
        } else {
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (there(j)) copy16(to + offset(j), from[m] + j * tpr * 16);
        }
        from[m] += step[m];
      }
    }
    copies_close();
    in += stage;
    if (in == slots) in = 0;
  }
  __device__ __forceinline__ void begin() {
    for (int i = 1; i < stages; ++i) fetch();
  }
  // Waits for the oldest row, then fetches one into the slot that the row before
  // it left; where the oldest is.
  __device__ __forceinline__ uint32_t next() {
    if (stages == 2) copies_left<0>();
    else if (stages == 3) copies_left<1>();
    else if (stages == 4) copies_left<2>();
    else copies_left<3>();
    if (SINGLE) group_barrier(group, tpr);
    const uint32_t at = first + out;
    out += stage;
    if (out == slots) out = 0;
    fetch();
    return at;
  }
  // What this thread has of matrix m's row, which starts at address `row`.
  __device__ __forceinline__ void get(uint32_t at, int m, const void* row, F2 (&v)[P]) const {
    at += m * matrix;
    if constexpr (!SINGLE) {
#pragma unroll
      for (int j = 0; j < NV; ++j) pairs_of<T>(ld_shared16(at + (there(j) ? offset(j) : 0)), v + j * (N / 2));
    } else {
      at += (uint32_t)((uintptr_t)row & 15u);
#pragma unroll
      for (int j = 0; j < NV; j += 2)
        v[j / 2] = f2(ld_shared1<T>(at + (there(j) ? offset(j) : 0)), ld_shared1<T>(at + (there(j + 1) ? offset(j + 1) : 0)));
    }
  }
  // The same into global memory, rounded; `to`: this thread's first vector.
  __device__ __forceinline__ void put(T* to, const F2 (&v)[P]) const {
    if constexpr (!SINGLE) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (there(j)) *reinterpret_cast<uint4*>((char*)to + j * tpr * 16) = packed<T>(v + j * (N / 2));
    } else {
#pragma unroll
      for (int j = 0; j < NV; j += 2) {
        const float2 x = split(v[j / 2]);
        if (there(j)) to[j * tpr] = from_f32<T>(x.x);
        if (there(j + 1)) to[(j + 1) * tpr] = from_f32<T>(x.y);
      }
    }
  }
  // A vector of columns, `none` where there is no such vector, 0 beside the row.
  template <typename W>
  __device__ __forceinline__ void columns(const void* p, float none, F2 (&v)[P]) const {
    float x[2 * P];
    const bool vec = !SINGLE && ((uintptr_t)p & 15u) == 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const W* w = (const W*)p + column(j);
#pragma unroll
      for (int i = 0; i < N; ++i) x[j * N + i] = there(j) ? none : 0.f;
      if (!p || !there(j)) continue;
      if (vec) {
        constexpr int K = N * sizeof(W) > 16 ? 16 / sizeof(W) : N;
#pragma unroll
        for (int q = 0; q < N; q += K) {
          const Pack<W, K> of = *reinterpret_cast<const Pack<W, K>*>(w + q);
#pragma unroll
          for (int i = 0; i < K; ++i) x[j * N + q + i] = to_f32(of.v[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[j * N + i] = to_f32(w[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = f2(x[2 * i], x[2 * i + 1]);
  }
};

// Sum over the lanes of a row: all, or the tpr (8 or 16) that have it.
__device__ __forceinline__ float lanes_sum(float x, int tpr) {
  if (tpr >= 32) x += __shfl_xor_sync(kAll, x, 16);
  if (tpr >= 16) x += __shfl_xor_sync(kAll, x, 8);
#pragma unroll
  for (int d = 4; d; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}

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

// ------------------------------------------------------------------ gradient
//
// With xh = (x - mean) / deviation and g = dy w:  dx = (g - mean(g) - xh mean(g
// xh)) / deviation (+ the gradient that reaches x beside the norm), and the
// columns' sums of dy xh and dy.  A CTA holds whole rows, its threads the
// columns' sums over the rows that pass through it; a second kernel adds the
// CTAs' sums, in order, or, of few rows, the CTAs of one cluster do.
//
// 8192 x 4096 bf16 with the residual's gradient: 50 us, 46 of them before the join; 5.4 TB/s, 80%
// of the copy bandwidth (39.5 us).  What is left is latency: 16 warps an SM at 120
// registers, a barrier for each row, 53% of the issue slots.  Loads when a row needs
// them: 112 us; by the ring 60; two values an instruction 54; sums across a warp by its
// halves and one round of loads in the join 50.  Launching the join early cost 2 us (its CTAs
// take the places of this kernel's last ones), CTAs of 1024 threads with 8 elements each
// 39.

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

bool even(const void* p, uint64_t ld, uint64_t size) { return !p || (((uintptr_t)p | ld * size) & 15u) == 0; }

constexpr uint32_t kSmem = 200 * 1024;
constexpr uint64_t kMostRow = 32 * 1024;  // bytes: of three matrices two fit

// How the threads of a CTA share rows: NV vectors in each, in groups of tpr threads.
// The group whose row costs the fewest instructions, by 14 instructions an element
// and 40 around them in each warp, 30 more where warps wait for each other (without
// these, 5120 bf16 values go to 20 warps, not 7: 134 us for 16384 rows, not 102; 20011 rows of 520
// binary32 to 5 warps, not one: 38 us for the gradient, not 24).
struct Shape {
  int cost = 0, nv = 0, tpr = 0;
  bool whole = false;
  void consider(int n, int vectors, uint64_t width) {
    const uint64_t per = (uint64_t)n * vectors;
    int t = (int)std::min<uint64_t>((width + per - 1) / per, 2 * kMostThreads);
    t = t <= 8 ? 8 : t <= 16 ? 16 : (t + 31) / 32 * 32;
    if (t > kMostThreads) return;
    const int c = t * (vectors * n * 14 + 40 + (t > 32 ? 30 : 0));
    if (cost && c >= cost) return;
    cost = c;
    nv = vectors;
    tpr = t;
    whole = per * t == width;
  }
};

// f(how rows lie, vectors of a thread, threads of a row), or wide() for rows that
// no CTA holds.
template <typename T, typename F, typename G>
purlin_status with_shape(bool aligned, uint64_t width, F f, G wide) {
  using std::integral_constant;
  constexpr integral_constant<Lie, Lie::kWhole> whole{};
  constexpr integral_constant<Lie, Lie::kPart> part{};
  constexpr integral_constant<Lie, Lie::kSingle> single{};
  constexpr integral_constant<int, 1> one{};
  constexpr integral_constant<int, 2> two{};
  constexpr integral_constant<int, 3> three{};
  constexpr integral_constant<int, 4> four{};
  constexpr integral_constant<int, 5> five{};
  constexpr int V = V16<T>;
  Shape s;
  if (aligned && width * sizeof(T) <= kMostRow) {
    if constexpr (V == 8) {
      for (int nv : {1, 2, 3}) s.consider(V, nv, width);
      if (s.nv == 3) return f(part, three, s.tpr);
    } else {
      for (int nv : {1, 2, 4}) s.consider(V, nv, width);
      if (width <= 32 * 5 * V) s.consider(V, 5, width);  // registers: only where it saves the barrier
      if (s.nv == 5) return f(part, five, s.tpr);
      if (s.nv == 4) return s.whole ? f(whole, four, s.tpr) : f(part, four, s.tpr);
    }
    if (s.nv == 2) return s.whole ? f(whole, two, s.tpr) : f(part, two, s.tpr);
    if (s.nv == 1) return s.whole ? f(whole, one, s.tpr) : f(part, one, s.tpr);
  }
  for (int nv : {4, 8, 16}) s.consider(1, nv, width);
  if (s.nv == 4) return f(single, four, s.tpr);
  if (s.nv == 8) return f(single, integral_constant<int, 8>(), s.tpr);
  if (s.nv == 16) return f(single, integral_constant<int, 16>(), s.tpr);
  return wide();
}

// The ring of a launch.
template <typename T>
Ring ring_of(Lie lie, uint64_t width, int tpr, int n) {
  Ring r = {};
  r.n = n;
  r.tpr = tpr;
  r.groups = kMostThreads / tpr;
  const uint64_t bytes = width * sizeof(T);
  r.granules = (uint32_t)((bytes + (lie == Lie::kSingle ? 30 : 0)) / 16);
  // as many rows under way as make 64 KiB, four at most (of 40 KiB, 16384 x 5120: 104 us
  // with one, 102 with two; of 65 KiB, 20011 x 520 binary32: 24.3 us with one, 25.5 with two)
  r.stages = 1;
  const uint32_t row = r.smem();
  for (r.stages = 2; r.stages < 5 && (uint32_t)(r.stages - 1) * row < 64 * 1024; ++r.stages) {
  }
  while (r.groups > 1 && r.smem() > kSmem) --r.groups;
  return r;
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

purlin_status launch_norm(const NormArgs& a, int dtype, int w_dtype, cudaStream_t s) {
  if (dtype == PL_F32) return w_dtype == PL_F32 ? norm_t<float, float>(a, s) : norm_t<float, bf16>(a, s);
  return w_dtype == PL_F32 ? norm_t<bf16, float>(a, s) : norm_t<bf16, bf16>(a, s);
}

purlin_status launch_norm_grad(const NormArgs& a, int dtype, int w_dtype, cudaStream_t s) {
  if (dtype == PL_F32) return w_dtype == PL_F32 ? norm_grad_t<float, float>(a, s) : norm_grad_t<float, bf16>(a, s);
  return w_dtype == PL_F32 ? norm_grad_t<bf16, float>(a, s) : norm_grad_t<bf16, bf16>(a, s);
}

}  // namespace pl
