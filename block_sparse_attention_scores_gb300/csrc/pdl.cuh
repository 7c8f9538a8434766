// Programmatic dependent launch: a kernel of a call is launched while the one
// before it still runs, sets itself up (barriers, TMEM, descriptors), and waits
// for that one's end and its writes before it touches global memory. What an
// earlier kernel may have written is read with ordinary loads (ld_in), not through
// the read-only path.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace msa {

// Waits for the kernel before this one in the stream, and everything before it.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel be launched once every block has come here (or ended).
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ int ld_in(const int* p) {
  int v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t ld_in(const uint32_t* p) { return (uint32_t)ld_in(reinterpret_cast<const int*>(p)); }
__device__ __forceinline__ float ld_in(const float* p) {
  return __int_as_float(ld_in(reinterpret_cast<const int*>(p)));
}
__device__ __forceinline__ float2 ld_in(const float2* p) {
  float2 v;
  asm volatile("ld.global.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_in(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ int4 ld_in(const int4* p) {
  const uint4 v = ld_in(reinterpret_cast<const uint4*>(p));
  return make_int4((int)v.x, (int)v.y, (int)v.z, (int)v.w);
}
__device__ __forceinline__ float4 ld_in(const float4* p) {
  const uint4 v = ld_in(reinterpret_cast<const uint4*>(p));
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                             Args&&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace msa
