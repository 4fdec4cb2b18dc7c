// Shared by the index-driven operators' kernels: rows as vectors of a width
// that the caller's alignment allows, conversion to binary32 and back, launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ops.h"
#include "purlin_atoms.cuh"

namespace pl {

// Every kernel here calls it before it writes, or reads what the stream's
// previous kernel writes: the launch may begin while that one drains, and its
// writes are visible after this.
__device__ __forceinline__ void op_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the stream's next kernel start as soon as every CTA here has started;
// its op_wait still waits for the end of this one.  Only after op_wait.
__device__ __forceinline__ void op_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// cluster > 1: in clusters of that many CTAs.
template <typename... P, typename... A>
inline purlin_status op_launch_cluster(int cluster, void (*fn)(P...), uint64_t grid, int threads, size_t smem,
                                       cudaStream_t s, const A&... args) {
  if (grid == 0) return PL_OK;
  if (grid > 0x7FFFFFFFull) return PL_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args...);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return PL_ERR_LAUNCH;
  }
  return PL_OK;
}

template <typename... P, typename... A>
inline purlin_status op_launch(void (*fn)(P...), uint64_t grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  return op_launch_cluster(1, fn, grid, threads, smem, s, args...);
}

// Lets `fn` take `need` bytes of dynamic shared memory, where that and its (at
// most 12 KiB) static memory are past the 48 KiB that every kernel may take: the
// limit is raised to `most`, the same each time.
inline purlin_status op_smem(const void* fn, size_t need, int most) {
  if (need <= 36 * 1024 || cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most) == cudaSuccess)
    return PL_OK;
  (void)cudaGetLastError();
  return PL_ERR_CUDA;
}

using bf16 = __nv_bfloat16;

// N elements of T, moved as one access of N * sizeof(T) bytes.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> ld_pack(const T* p) {
  Pack<T, N> r;
  if constexpr (sizeof(T) * N == 16) {
    uint4 u;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    memcpy(&r, &u, 16);
  } else if constexpr (sizeof(T) * N == 8) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    memcpy(&r, &u, 8);
  } else if constexpr (sizeof(T) * N == 4) {
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(p));
    memcpy(&r, &u, 4);
  } else {
    const unsigned short u = __ldg(reinterpret_cast<const unsigned short*>(p));
    memcpy(&r, &u, 2);
  }
  return r;
}

// 16 bytes at p, or zeros where `on` is false: one predicated load.  Written as
// a branch around a load and one around its use, the compiler joins the two,
// and each load then waits for the one before (150 us instead of 71 for a sum of
// 6 rows of 8 KiB for each of 8192 tokens).  KEPT: into the L1 too.  WRITTEN: of
// memory that this kernel writes, not through the read-only path.
enum class Ld { kOnce, kKept, kWritten };
template <Ld HOW = Ld::kOnce>
__device__ __forceinline__ uint4 ld16_if(const void* p, bool on) {
  uint4 v;
#define PL_LD16_IF(op)                                                                                               \
  asm volatile(                                                                                                      \
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"          \
      "mov.u32 %3, 0;\n\t@q " op " {%0,%1,%2,%3}, [%4];\n\t}"                                                       \
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)                                                               \
      : "l"(p), "r"((uint32_t)on))
  if constexpr (HOW == Ld::kOnce) PL_LD16_IF("ld.global.nc.L1::no_allocate.v4.u32");
  else if constexpr (HOW == Ld::kKept) PL_LD16_IF("ld.global.nc.v4.u32");
  else PL_LD16_IF("ld.global.v4.u32");
#undef PL_LD16_IF
  return v;
}

// One element at p, or zero: predicated too.
__device__ __forceinline__ float ld1_if(const float* p, bool on) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\tmov.u32 %0, 0;\n\t@q ld.global.nc.u32 %0, [%1];\n\t}"
               : "=&r"(v)
               : "l"(p), "r"((uint32_t)on));
  return __uint_as_float(v);
}
__device__ __forceinline__ float ld1_if(const bf16* p, bool on) {
  unsigned short v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\tmov.u16 %0, 0;\n\t@q ld.global.nc.u16 %0, [%1];\n\t}"
               : "=&h"(v)
               : "l"(p), "r"((uint32_t)on));
  return __uint_as_float((uint32_t)v << 16);
}

// Nothing that uses r is moved before this, nor what is written before it
// behind: loads above stay together, all in flight before the first is used.
template <typename T, int N>
__device__ __forceinline__ void pin(Pack<T, N>& r) {
  if constexpr (sizeof(T) * N == 16) {
    uint4 u;
    memcpy(&u, &r, 16);
    asm volatile("" : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w));
    memcpy(&r, &u, 16);
  }
}

template <typename T, int N, Ld HOW = Ld::kOnce>
__device__ __forceinline__ Pack<T, N> ld_pack_if(const T* p, bool on) {
  Pack<T, N> r;
  if constexpr (sizeof(T) * N == 16) {
    const uint4 u = ld16_if<HOW>(p, on);
    memcpy(&r, &u, 16);
  } else {
    static_assert(HOW == Ld::kOnce);
    memset(&r, 0, sizeof r);
    if (on) r = ld_pack<T, N>(p);
  }
  return r;
}

// Rows are moved in 16-byte vectors that are aligned at their destination.  V:
// elements of one.  SHIFT: the source need not be aligned with it; a vector is
// then cut from the two aligned granules that hold its bytes (both of which
// hold bytes of the row).
template <typename T>
constexpr int V16 = 16 / sizeof(T);
template <typename T, bool SHIFT>
__device__ __forceinline__ Pack<T, V16<T>> ld_row_if(const T* p, bool on) {
  Pack<T, V16<T>> r;
  uint4 u;
  if (!SHIFT) {
    u = ld16_if(p, on);
  } else {
    const uint32_t m = (uint32_t)((uintptr_t)p & 15u);
    const char* a = (const char*)p - m;
    const uint4 A = ld16_if<Ld::kKept>(a, on), B = ld16_if<Ld::kKept>(a + 16, on && m);
    u = m ? window16(A, B, m) : A;
  }
  memcpy(&r, &u, 16);
  return r;
}

// A row of `width` elements at a destination: `head` elements before its first
// aligned vector, nv vectors, and the rest.
struct Cut {
  uint32_t head, beside;  // elements before, and before and behind the vectors
  uint64_t nv;
  // the i-th element beside the vectors
  template <int V>
  __device__ __forceinline__ uint64_t at(uint32_t i) const {
    return i < head ? i : i + nv * V;
  }
};
template <typename T, bool SHIFT>
__device__ __forceinline__ Cut cut_of(const T* dst, uint64_t width) {
  if (!SHIFT) return {0, 0, width / V16<T>};
  const uint32_t off = (uint32_t)((uintptr_t)dst & 15u) / sizeof(T), gap = off ? V16<T> - off : 0;
  const uint32_t head = (uint64_t)gap < width ? gap : (uint32_t)width;
  const uint64_t nv = (width - head) / V16<T>;
  return {head, (uint32_t)(width - nv * V16<T>), nv};
}

template <typename T, int N>
__device__ __forceinline__ void st_pack(T* p, const Pack<T, N>& r) {
  *reinterpret_cast<Pack<T, N>*>(p) = r;
}

// The same, evict-first: data that nobody here reads again.
template <typename T, int N>
__device__ __forceinline__ void st_pack_once(T* p, const Pack<T, N>& r) {
  if constexpr (sizeof(T) * N == 16) {
    __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&r));
  } else if constexpr (sizeof(T) * N == 8) {
    __stcs(reinterpret_cast<uint2*>(p), *reinterpret_cast<const uint2*>(&r));
  } else {
    st_pack<T, N>(p, r);
  }
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x) {
  return __float2bfloat16_rn(x);
}

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> zero_pack() {
  Pack<T, N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) r.v[i] = from_f32<T>(0.f);
  return r;
}

// Two binary32 values that one instruction takes at once, each rounded as alone.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float both(F2 a) {
  const float2 s = split(a);
  return s.x + s.y;
}

// 16 bytes of T as pairs, and back (bf16: rounded two at a time).
__device__ __forceinline__ F2 pair_of(uint32_t bf16x2) {
  return f2(__uint_as_float(bf16x2 << 16), __uint_as_float(bf16x2 & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t bf16x2_of(F2 a) {
  const float2 s = split(a);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(s.y), "f"(s.x));
  return r;
}
template <typename T>
__device__ __forceinline__ void pairs_of(uint4 u, F2* p) {
  if constexpr (sizeof(T) == 2) {
    p[0] = pair_of(u.x);
    p[1] = pair_of(u.y);
    p[2] = pair_of(u.z);
    p[3] = pair_of(u.w);
  } else {
    p[0] = f2(__uint_as_float(u.x), __uint_as_float(u.y));
    p[1] = f2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
}
template <typename T>
__device__ __forceinline__ uint4 packed(const F2* p) {
  if constexpr (sizeof(T) == 2) return make_uint4(bf16x2_of(p[0]), bf16x2_of(p[1]), bf16x2_of(p[2]), bf16x2_of(p[3]));
  const float2 a = split(p[0]), b = split(p[1]);
  return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
}

__device__ __forceinline__ void op_status(uint32_t* status, uint32_t what) { atomicCAS(status, 0u, what); }

constexpr int kRowThreads = 256;

// Groups of threads that cover a row of nv vectors in the fewest rounds of at
// most 256, with as few idle threads as whole warps allow; CTAs of 256 threads.
struct RowShape {
  int tpt, per;
  template <typename T>
  static RowShape of(uint64_t width, bool shift) {  // vectors, and the elements beside them
    return RowShape(width / V16<T> + (shift ? 2 * (V16<T> - 1) : 0));
  }
  explicit RowShape(uint64_t nv) {
    const uint64_t rounds = std::max<uint64_t>(1, (nv + kRowThreads - 1) / kRowThreads);
    tpt = std::max(32, (int)((nv + rounds * 32 - 1) / (rounds * 32)) * 32);
    per = kRowThreads / tpt;
  }
  uint64_t ctas(uint64_t tokens, int u) const { return (tokens + per * u - 1) / (per * u); }
};
// Several tokens per group pay off where the CTAs still fill the SMs twice (1
// pick of 2048 bf16 values, one token at a time and four: 300 tokens 2.4 and 3.0
// us, 1300 tokens 4.3 and 3.6; embedding the same, 300: 2.4, 2.6, 5000: 8.8, 7.3).
constexpr uint64_t kManyCtas = 2 * 152;

}  // namespace pl
