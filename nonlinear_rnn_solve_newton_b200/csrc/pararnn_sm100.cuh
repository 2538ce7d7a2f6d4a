// pararnn_sm100.cuh -- what several kernels share of sm_100: pairs of fp32, and launches
// that overlap.
#pragma once

#include <cuda_runtime.h>

namespace pararnn {

// Two fp32 operations in one instruction, on a pair of neighbouring registers.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair2(float x, float y) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ void unpair2(f32x2 d, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(d));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A kernel launched by launch_behind starts while the last CTAs of the kernel ahead of it
// in the stream end, not after.  It touches nothing that the other kernel reads or
// writes before wait_for_launch_before, which returns once that kernel has ended and its
// writes are there (in a kernel launched otherwise: at once).  The join behind a layer
// norm's backward pass and those between the walks of linear attention gain 1 to 3 us
// each.  A trigger at the start of the kernel ahead (griddepcontrol.launch_dependents)
// takes that back: 262144 x 128 backward 46.4 us with it, 43.8 without, 44.8 launched
// plainly.
__device__ __forceinline__ void wait_for_launch_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t st, const A&... args) {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pararnn
