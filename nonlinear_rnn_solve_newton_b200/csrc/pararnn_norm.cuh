// pararnn_norm.cuh -- layer norm over the last axis, forward and backward.
//
//   mean = sum(x) / D,  rstd = (sum((x - mean)^2) / D + eps)^(-1/2)
//   y = (x - mean) rstd w + b
//   g = dy w,  xh = (x - mean) rstd
//   dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum dy xh,  db = sum dy
//
// All sums are fp32; the variance is the two-pass one (mean first).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pararnn {

struct NormParams {
  const void* x;    // [M, D] rows at stride sx
  const void* dy;   // backward: [M, D], rows at stride sdy
  const float* w;   // [D] or NULL (= 1)
  const float* b;   // [D] or NULL (= 0)
  void* y;          // forward: y; backward: dx; rows dense
  float* mean;      // [M]
  float* rstd;      // [M]
  float* part;      // backward: [2][nparts][D] partial sums of dw and db
  float* dw;        // [D]
  float* db;        // [D]
  long long M, sx, sdy;
  int D, nparts;
  float eps;
};

__device__ __forceinline__ float norm_load(const float* p) { return *p; }
__device__ __forceinline__ float norm_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void norm_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void norm_store(__nv_bfloat16* p, float v) {
  *p = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// One warp per row.
template <typename TX, typename TY>
__global__ void __launch_bounds__(256) pararnn_norm_kernel(const __grid_constant__ NormParams p) {
  const long long row = blockIdx.x * 8LL + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= p.M) return;
  const TX* x = static_cast<const TX*>(p.x) + row * p.sx;
  TY* y = static_cast<TY*>(p.y) + row * p.D;
  float s = 0.0f;
  for (int d = lane; d < p.D; d += 32) s += norm_load(x + d);
  const float mean = warp_sum(s) / (float)p.D;
  s = 0.0f;
  for (int d = lane; d < p.D; d += 32) {
    const float c = norm_load(x + d) - mean;
    s = fmaf(c, c, s);
  }
  const float rstd = 1.0f / sqrtf(warp_sum(s) / (float)p.D + p.eps);
  for (int d = lane; d < p.D; d += 32) {
    const float xh = (norm_load(x + d) - mean) * rstd;
    norm_store(y + d, fmaf(xh, p.w ? p.w[d] : 1.0f, p.b ? p.b[d] : 0.0f));
  }
  if (lane == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
}

// dx, one warp per row.
template <typename TX, typename TY>
__global__ void __launch_bounds__(256)
    pararnn_norm_dx_kernel(const __grid_constant__ NormParams p) {
  const long long row = blockIdx.x * 8LL + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= p.M) return;
  const TX* x = static_cast<const TX*>(p.x) + row * p.sx;
  const TY* dy = static_cast<const TY*>(p.dy) + row * p.sdy;
  TX* dx = static_cast<TX*>(p.y) + row * p.D;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float sg = 0.0f, sgx = 0.0f;
  for (int d = lane; d < p.D; d += 32) {
    const float g = norm_load(dy + d) * (p.w ? p.w[d] : 1.0f);
    sg += g;
    sgx = fmaf(g, (norm_load(x + d) - mean) * rstd, sgx);
  }
  const float mg = warp_sum(sg) / (float)p.D, mgx = warp_sum(sgx) / (float)p.D;
  for (int d = lane; d < p.D; d += 32) {
    const float g = norm_load(dy + d) * (p.w ? p.w[d] : 1.0f);
    const float xh = (norm_load(x + d) - mean) * rstd;
    norm_store(dx + d, rstd * (g - mg - xh * mgx));
  }
}

// Column sums of one slice of rows: thread = column.
template <typename TX, typename TY>
__global__ void __launch_bounds__(128)
    pararnn_norm_dw_kernel(const __grid_constant__ NormParams p) {
  const int d = blockIdx.x * 128 + threadIdx.x;
  if (d >= p.D) return;
  const long long lo = p.M * blockIdx.y / p.nparts, hi = p.M * (blockIdx.y + 1) / p.nparts;
  float sw = 0.0f, sb = 0.0f;
  for (long long r = lo; r < hi; ++r) {
    const float dy = norm_load(static_cast<const TY*>(p.dy) + r * p.sdy + d);
    const float xh = (norm_load(static_cast<const TX*>(p.x) + r * p.sx + d) - p.mean[r]) * p.rstd[r];
    sw = fmaf(dy, xh, sw);
    sb += dy;
  }
  p.part[(long long)blockIdx.y * p.D + d] = sw;
  p.part[(long long)(p.nparts + blockIdx.y) * p.D + d] = sb;
}

// The slices' sums, joined in a fixed order.
__global__ void pararnn_norm_join_kernel(const __grid_constant__ NormParams p) {
  const int d = blockIdx.x * blockDim.x + threadIdx.x;
  if (d >= p.D) return;
  float sw = 0.0f, sb = 0.0f;
  for (int i = 0; i < p.nparts; ++i) {
    sw += p.part[(long long)i * p.D + d];
    sb += p.part[(long long)(p.nparts + i) * p.D + d];
  }
  p.dw[d] = sw;
  p.db[d] = sb;
}

}  // namespace pararnn
