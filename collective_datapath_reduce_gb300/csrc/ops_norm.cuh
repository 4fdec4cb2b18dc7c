// Shared by the layer norm's kernels: rows that pass through a CTA, and how its
// threads share them.
#pragma once

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
// 16 bytes of shared memory, or zeros where `on` is false.
__device__ __forceinline__ uint4 ld_shared16_if(uint32_t at, bool on) {
  uint4 u;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
      "mov.u32 %3, 0;\n\t@q ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "=&r"(u.x), "=&r"(u.y), "=&r"(u.z), "=&r"(u.w)
      : "r"(at), "r"((uint32_t)on)
      : "memory");
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
// pairs.  A vector beside the row is zeros (kSingle: the row's first element), and
// counts 0 times.  No thread reads what another's copy brings, but for kSingle, whose
// threads wait for each other first.
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
      for (int j = 0; j < NV; ++j) pairs_of<T>(ld_shared16_if(at + offset(j), there(j)), v + j * (N / 2));
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

inline bool even(const void* p, uint64_t ld, uint64_t size) { return !p || (((uintptr_t)p | ld * size) & 15u) == 0; }

constexpr uint32_t kSmem = 200 * 1024;

// How the threads of a CTA share rows: NV vectors in each, in groups of tpr threads.
// The group whose row costs the fewest instructions, by 14 instructions an element
// and 40 around them in each warp, 30 more where warps wait for each other.  Without the 40
// and 30, 5120 bf16 values go to 10 warps, not 7 (16384 rows with a residual: 125 us, not 100),
// and 520 binary32 values to 5 warps, not one (20011 rows: 39 us, not 12; the gradient 44, not
// 23).  What 512 / tpr threads leave idle does not count, and should: 7168 and 8192 bf16 values
// go to 10 and 11 warps, alone on their SM (8192 rows with a residual: 85 and 89 us, the gradient
// 135 and 142), where 14 and 16 warps with two vectors a thread take 78 and 83, 87 and 94.
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
  if (aligned) {
    if constexpr (V == 8) {
      for (int nv : {1, 2, 3}) s.consider(V, nv, width);
      if (s.nv == 3) return f(part, three, s.tpr);
    } else {
      for (int nv : {1, 2, 4}) s.consider(V, nv, width);
      // five, for their registers, only where a warp at most then has the row (160 / 320 / 640 values, 64 MB of
      // them: 17.9 / 18.4 / 19.0 us, without 23.6 / 24.0 / 34.8; the gradient 32.4 / 32.3 / 32.8, without 36.9 / 36.6 / 41.4)
      if (width <= 32 * 5 * V) s.consider(V, 5, width);
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
  // whole warps, whose lanes vote and shuffle together (binary32 rows of 136 to 160 values, three matrices)
  const int step = std::max(1, 32 / tpr);
  while (r.groups > step && r.smem() > kSmem) r.groups -= step;
  return r;
}

}  // namespace
}  // namespace pl
