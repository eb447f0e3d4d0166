// Rows taken 16 bytes at a time: values of a vector as floats, and back.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "tg_ptx.cuh"

namespace tg {

template <typename T> struct Vec16;
template <> struct Vec16<float> {
  static constexpr int E = 4;  // values of a vector
  static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y); f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <> struct Vec16<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float* f) {
    f[0] = ptx::bf16lo(u.x); f[1] = ptx::bf16hi(u.x); f[2] = ptx::bf16lo(u.y); f[3] = ptx::bf16hi(u.y);
    f[4] = ptx::bf16lo(u.z); f[5] = ptx::bf16hi(u.z); f[6] = ptx::bf16lo(u.w); f[7] = ptx::bf16hi(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                      ptx::pack_bf16x2(f[6], f[7]));
  }
};

inline bool aligned_16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The elements of a row before its first 16-byte boundary, at most n.
template <typename T>
__device__ __forceinline__ int row_lead(const T* row, int n) {
  return min(n, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T));
}

// For a kernel that is launched before the one ahead of it has ended.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launches a kernel that may start while the one ahead of it in the stream still runs; it waits itself
// (wait_for_previous).
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace tg
