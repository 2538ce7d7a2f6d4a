// norm.cu -- C ABI of layer norm (declared in include/pararnn.h): argument
// validation and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pararnn.h"
#include "pararnn_norm.cuh"

namespace pararnn {
namespace {

constexpr int kNormSms = 148;

// Columns are counted in int, and a thread's next column is up to 1024 beyond the row.
constexpr int64_t kNormMaxCols = 1LL << 30;

bool norm_sizes_ok(int64_t M, int64_t D) {
  return M >= 0 && D > 0 && D <= kNormMaxCols && M < (1LL << 31);
}

bool norm_aligned(const void* p, pararnn_dtype_t t) {
  return ((uintptr_t)p % (t == PARARNN_F32 ? 4 : 2)) == 0;
}

bool norm_dtype_ok(pararnn_dtype_t t) { return t == PARARNN_F32 || t == PARARNN_BF16; }

// Most CTAs of the backward pass: 8 a SM of small ones, and no more partial sums than
// 8 CTAs of 1024 columns a SM would write (at M = 16384, D = 4096 they are 4% of the
// traffic).
int norm_max_parts(int64_t D) {
  const int64_t n = (int64_t)kNormSms * 8 * 1024 / D;
  return (int)(n > kNormSms * 8 ? kNormSms * 8 : (n < kNormSms ? kNormSms : n));
}

size_t norm_ws(int64_t M, int64_t D) {
  const int64_t most = norm_max_parts(D);
  if (M <= 1) return 256;  // needs none
  return ((size_t)2 * (M < most ? M : most) * D * 4 + 255) / 256 * 256 + 256;
}

// How a row is held.  Whole warps hold up to kWarpGroups groups a lane, a CTA the rest;
// rows that 512 threads cannot hold are read more than once.
struct NormShape {
  bool vec, cta, fits;
  int tpr, groups;  // threads of a row, groups a thread
};

bool norm_vec(const void* p, pararnn_dtype_t t, int64_t stride, int64_t M) {
  const int unit = t == PARARNN_F32 ? 4 : 8;
  return ((uintptr_t)p % 16) == 0 && (M <= 1 || stride % unit == 0);
}

NormShape norm_shape(bool vec, int64_t D, int warp_groups, int cta_groups, int most_groups) {
  NormShape s = {vec, false, true, 1, warp_groups};
  const int64_t n = vec ? D / 8 : D;  // groups of a row
  if (n <= 32 * warp_groups) {
    while ((int64_t)s.tpr * warp_groups < n) s.tpr *= 2;
    while (s.groups > 1 && (int64_t)s.tpr * (s.groups / 2) >= n) s.groups /= 2;
    return s;
  }
  s.cta = true;
  s.groups = cta_groups;
  while (s.groups < most_groups && 512LL * s.groups < n) s.groups *= 2;
  s.tpr = 64;
  while (s.tpr < 512 && (int64_t)s.tpr * s.groups < n) s.tpr *= 2;
  s.fits = (int64_t)s.tpr * s.groups >= n;
  return s;
}

template <typename TX, typename TY, int VEC, int G>
void norm_fwd_go(NormParams& np, const NormShape& sh, cudaStream_t st) {
  np.tpr = sh.tpr;
  if (sh.cta) {  // always with the most groups
    if constexpr (VEC == 1 || G == 4)
      pararnn_norm_kernel<TX, TY, VEC, G, true><<<(unsigned)np.M, sh.tpr, 0, st>>>(np);
  } else {
    const long long rows = (long long)(kNormThreads / 32) * (32 / sh.tpr);
    pararnn_norm_kernel<TX, TY, VEC, G, false>
        <<<(unsigned)((np.M + rows - 1) / rows), kNormThreads, 0, st>>>(np);
  }
}

template <typename TX, typename TY>
void norm_fwd(NormParams& np, bool vec, cudaStream_t st) {
  // up to 4 groups of 8 a lane (128 bytes of fp32), 16 single elements
  const NormShape sh = vec ? norm_shape(true, np.D, 4, 4, 4) : norm_shape(false, np.D, 16, 16, 16);
  if (!sh.fits) {
    pararnn_norm_long_kernel<TX, TY><<<(unsigned)np.M, 1024, 0, st>>>(np);
  } else if (vec) {
    if (sh.groups == 4)
      norm_fwd_go<TX, TY, 8, 4>(np, sh, st);
    else if (sh.groups == 2)
      norm_fwd_go<TX, TY, 8, 2>(np, sh, st);
    else
      norm_fwd_go<TX, TY, 8, 1>(np, sh, st);
  } else {
    norm_fwd_go<TX, TY, 1, 16>(np, sh, st);
  }
}

template <typename TX, typename TY, int VEC, int G, int R>
void norm_bwd_go(NormParams& np, const NormShape& sh, cudaStream_t st) {
  np.tpr = sh.tpr;
  const long long rows = sh.cta ? 1 : (long long)(kNormThreads / 32) * (32 / sh.tpr);
  // enough CTAs to fill the SMs (512 threads of a CTA-wide row, or two 8-warp CTAs), each
  // with R rows at a time
  long long most = sh.cta ? (long long)kNormSms * (512 / sh.tpr) : 2LL * kNormSms;
  if (most > norm_max_parts(np.D)) most = norm_max_parts(np.D);
  const long long want = (np.M + rows - 1) / rows;
  np.nparts = (int)(want < most ? want : most);
  // vectors are held by whole warps one group a lane
  if (sh.cta)
    pararnn_norm_bwd_kernel<TX, TY, VEC, G, R, true><<<np.nparts, sh.tpr, 0, st>>>(np);
  else if constexpr (VEC == 1 || G == 1)
    pararnn_norm_bwd_kernel<TX, TY, VEC, G, R, false>
        <<<np.nparts, kNormThreads, 8 * (size_t)np.D, st>>>(np);
}

void norm_join(const NormParams& np, cudaStream_t st) {
  launch_behind(pararnn_norm_join_kernel, dim3((unsigned)((np.D + 31) / 32)),
                dim3(32 * kNormSlices), 0, st, np);
}

template <typename TX, typename TY>
void norm_bwd(NormParams& np, bool vec, cudaStream_t st) {
  const NormShape sh = vec ? norm_shape(true, np.D, 1, 1, 4) : norm_shape(false, np.D, 16, 16, 16);
  if (!sh.fits) {
    np.nparts = (int)(np.M < kNormSms ? np.M : kNormSms);
    pararnn_norm_long_dx_kernel<TX, TY><<<(unsigned)np.M, 1024, 0, st>>>(np);
    pararnn_norm_long_dw_kernel<TX, TY>
        <<<dim3((unsigned)((np.D + 127) / 128), (unsigned)np.nparts), 128, 0, st>>>(np);
  } else if (vec) {
    if (sh.groups == 4)
      norm_bwd_go<TX, TY, 8, 4, 1>(np, sh, st);
    else if (sh.groups == 2)
      norm_bwd_go<TX, TY, 8, 2, 1>(np, sh, st);
    else
      norm_bwd_go<TX, TY, 8, 1, 2>(np, sh, st);
  } else {
    norm_bwd_go<TX, TY, 1, 16, 1>(np, sh, st);
  }
  // one part went straight to dweight and dbias; a single row has no workspace
  if (np.nparts > 1) norm_join(np, st);
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
  const bool vec = D % 8 == 0 && norm_vec(x, x_dtype, x_stride, M) &&
                   norm_vec(y, y_dtype, D, M) && norm_vec(weight, PARARNN_F32, 0, 0) &&
                   norm_vec(bias, PARARNN_F32, 0, 0);
  if (x_dtype == PARARNN_F32) {
    if (y_dtype == PARARNN_F32)
      norm_fwd<float, float>(np, vec, st);
    else
      norm_fwd<float, __nv_bfloat16>(np, vec, st);
  } else {
    if (y_dtype == PARARNN_F32)
      norm_fwd<__nv_bfloat16, float>(np, vec, st);
    else
      norm_fwd<__nv_bfloat16, __nv_bfloat16>(np, vec, st);
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
  // one row, one partial sum: it is the result
  if (M > 1 && (!ws || ws_bytes < norm_ws(M, D) || ((uintptr_t)ws % 256) != 0))
    return PARARNN_ERR_WORKSPACE;
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
  const bool vec = D % 8 == 0 && norm_vec(x, x_dtype, x_stride, M) &&
                   norm_vec(dy, dy_dtype, dy_stride, M) && norm_vec(dx, x_dtype, D, M) &&
                   norm_vec(weight, PARARNN_F32, 0, 0);
  if (x_dtype == PARARNN_F32) {
    if (dy_dtype == PARARNN_F32)
      norm_bwd<float, float>(np, vec, st);
    else
      norm_bwd<float, __nv_bfloat16>(np, vec, st);
  } else {
    if (dy_dtype == PARARNN_F32)
      norm_bwd<__nv_bfloat16, float>(np, vec, st);
    else
      norm_bwd<__nv_bfloat16, __nv_bfloat16>(np, vec, st);
  }
  return cudaGetLastError() == cudaSuccess ? PARARNN_OK : PARARNN_ERR_CUDA;
}
