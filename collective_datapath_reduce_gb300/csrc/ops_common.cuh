// Shared by the index-driven operators' kernels: rows as vectors of a width
// that the caller's alignment allows, conversion to binary32 and back, launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ops.h"

namespace pl {

// The start of every kernel here: the launch may begin while the previous
// kernel of the stream drains; its writes are visible after this.
__device__ __forceinline__ void op_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
inline purlin_status op_launch(void (*fn)(P...), uint64_t grid, int threads, size_t smem, cudaStream_t s, A... args) {
  if (grid == 0) return PL_OK;
  if (grid > 0x7FFFFFFFull) return PL_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args...);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return PL_ERR_LAUNCH;
  }
  return PL_OK;
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

template <typename T, int N>
__device__ __forceinline__ void st_pack(T* p, const Pack<T, N>& r) {
  *reinterpret_cast<Pack<T, N>*>(p) = r;
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

__device__ __forceinline__ void op_status(uint32_t* status, uint32_t what) { atomicCAS(status, 0u, what); }

// Widest access (16, 8, 4, 2 bytes) that divides every address and byte
// count or stride or-ed into `bits`.
inline int vec_bytes(uint64_t bits) {
  const uint64_t low = bits & (~bits + 1);
  return low == 0 || low > 16 ? 16 : (int)low;
}

// Runs f(integral_constant N) for the N elements of T that fit `bytes`.
template <typename T, typename F>
inline purlin_status with_vec(int bytes, F f) {
  const int n = bytes / (int)sizeof(T);
  if constexpr (sizeof(T) == 2)
    if (n >= 8) return f(std::integral_constant<int, 8>());
  if (n >= 4) return f(std::integral_constant<int, 4>());
  if (n >= 2) return f(std::integral_constant<int, 2>());
  return f(std::integral_constant<int, 1>());
}

}  // namespace pl
