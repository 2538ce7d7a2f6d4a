// norm.cu -- C ABI of layer norm (declared in include/pararnn.h): argument
// validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pararnn.h"
#include "pararnn_norm.cuh"

namespace pararnn {
namespace {

constexpr int kNormParts = 148;

bool norm_sizes_ok(int64_t M, int64_t D) {
  return M >= 0 && D > 0 && D < (1LL << 31) && M < (1LL << 31) * 4 && M < (1LL << 62) / D;
}

bool norm_aligned(const void* p, pararnn_dtype_t t) {
  return ((uintptr_t)p % (t == PARARNN_F32 ? 4 : 2)) == 0;
}

bool norm_dtype_ok(pararnn_dtype_t t) { return t == PARARNN_F32 || t == PARARNN_BF16; }

int norm_parts(int64_t M) { return (int)(M < 1 ? 1 : (M < kNormParts ? M : kNormParts)); }

size_t norm_ws(int64_t M, int64_t D) {
  return ((size_t)2 * norm_parts(M) * D * 4 + 255) / 256 * 256;
}

template <typename TX, typename TY>
void norm_bwd_launch(const NormParams& np, cudaStream_t st) {
  pararnn_norm_dx_kernel<TX, TY><<<(unsigned)((np.M + 7) / 8), 256, 0, st>>>(np);
  pararnn_norm_dw_kernel<TX, TY><<<dim3((unsigned)((np.D + 127) / 128), (unsigned)np.nparts), 128,
                                   0, st>>>(np);
  pararnn_norm_join_kernel<<<(unsigned)((np.D + 127) / 128), 128, 0, st>>>(np);
}

}  // namespace
}  // namespace pararnn

using namespace pararnn;

extern "C" pararnn_status_t pararnn_layer_norm(const void* x, pararnn_dtype_t x_dtype,
                                               int64_t x_stride, const float* weight,
                                               const float* bias, void* y,
                                               pararnn_dtype_t y_dtype, float* mean, float* rstd,
                                               int64_t M, int64_t D, float eps, void* stream) {
  if (!norm_sizes_ok(M, D) || !norm_dtype_ok(x_dtype) || !norm_dtype_ok(y_dtype))
    return PARARNN_ERR_INVALID_ARGUMENT;
  if (!(eps >= 0.0f) || std::isinf(eps)) return PARARNN_ERR_INVALID_ARGUMENT;
  if (M == 0) return PARARNN_OK;
  if (!x || !y || !mean || !rstd || x_stride < 0 || x_stride >= (1LL << 40))
    return PARARNN_ERR_INVALID_ARGUMENT;
  if (!norm_aligned(x, x_dtype) || !norm_aligned(y, y_dtype) ||
      !norm_aligned(weight, PARARNN_F32) || !norm_aligned(bias, PARARNN_F32) ||
      !norm_aligned(mean, PARARNN_F32) || !norm_aligned(rstd, PARARNN_F32))
    return PARARNN_ERR_INVALID_ARGUMENT;
  NormParams np = {};
  np.x = x;
  np.w = weight;
  np.b = bias;
  np.y = y;
  np.mean = mean;
  np.rstd = rstd;
  np.M = M;
  np.D = (int)D;
  np.sx = x_stride;
  np.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)((M + 7) / 8);
  if (x_dtype == PARARNN_F32) {
    if (y_dtype == PARARNN_F32)
      pararnn_norm_kernel<float, float><<<grid, 256, 0, st>>>(np);
    else
      pararnn_norm_kernel<float, __nv_bfloat16><<<grid, 256, 0, st>>>(np);
  } else {
    if (y_dtype == PARARNN_F32)
      pararnn_norm_kernel<__nv_bfloat16, float><<<grid, 256, 0, st>>>(np);
    else
      pararnn_norm_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 256, 0, st>>>(np);
  }
  return cudaGetLastError() == cudaSuccess ? PARARNN_OK : PARARNN_ERR_CUDA;
}

extern "C" size_t pararnn_layer_norm_workspace_size(int64_t M, int64_t D) {
  return norm_sizes_ok(M, D) ? norm_ws(M, D) : 0;
}

extern "C" pararnn_status_t pararnn_layer_norm_backward(
    const void* dy, pararnn_dtype_t dy_dtype, int64_t dy_stride, const void* x,
    pararnn_dtype_t x_dtype, int64_t x_stride, const float* weight, const float* mean,
    const float* rstd, void* dx, float* dweight, float* dbias, int64_t M, int64_t D, void* ws,
    size_t ws_bytes, void* stream) {
  if (!norm_sizes_ok(M, D) || !norm_dtype_ok(x_dtype) || !norm_dtype_ok(dy_dtype))
    return PARARNN_ERR_INVALID_ARGUMENT;
  if (!dweight || !dbias || !norm_aligned(dweight, PARARNN_F32) ||
      !norm_aligned(dbias, PARARNN_F32))
    return PARARNN_ERR_INVALID_ARGUMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (M == 0)
    return cudaMemsetAsync(dweight, 0, 4 * (size_t)D, st) == cudaSuccess &&
                   cudaMemsetAsync(dbias, 0, 4 * (size_t)D, st) == cudaSuccess
               ? PARARNN_OK
               : PARARNN_ERR_CUDA;
  if (!dy || !x || !dx || !mean || !rstd || x_stride < 0 || dy_stride < 0 ||
      x_stride >= (1LL << 40) || dy_stride >= (1LL << 40))
    return PARARNN_ERR_INVALID_ARGUMENT;
  if (!norm_aligned(x, x_dtype) || !norm_aligned(dx, x_dtype) || !norm_aligned(dy, dy_dtype) ||
      !norm_aligned(weight, PARARNN_F32) || !norm_aligned(mean, PARARNN_F32) ||
      !norm_aligned(rstd, PARARNN_F32))
    return PARARNN_ERR_INVALID_ARGUMENT;
  if (!ws || ws_bytes < norm_ws(M, D) || ((uintptr_t)ws % 256) != 0) return PARARNN_ERR_WORKSPACE;
  NormParams np = {};
  np.x = x;
  np.dy = dy;
  np.w = weight;
  np.y = dx;
  np.mean = const_cast<float*>(mean);
  np.rstd = const_cast<float*>(rstd);
  np.part = static_cast<float*>(ws);
  np.dw = dweight;
  np.db = dbias;
  np.M = M;
  np.D = (int)D;
  np.sx = x_stride;
  np.sdy = dy_stride;
  np.nparts = norm_parts(M);
  if (x_dtype == PARARNN_F32) {
    if (dy_dtype == PARARNN_F32)
      norm_bwd_launch<float, float>(np, st);
    else
      norm_bwd_launch<float, __nv_bfloat16>(np, st);
  } else {
    if (dy_dtype == PARARNN_F32)
      norm_bwd_launch<__nv_bfloat16, float>(np, st);
    else
      norm_bwd_launch<__nv_bfloat16, __nv_bfloat16>(np, st);
  }
  return cudaGetLastError() == cudaSuccess ? PARARNN_OK : PARARNN_ERR_CUDA;
}
