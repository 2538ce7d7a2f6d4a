// pararnn_norm.cuh -- layer norm over the last axis, forward and backward.
//
//   mean = sum(x) / D,  rstd = (sum((x - mean)^2) / D + eps)^(-1/2)
//   y = (x - mean) rstd w + b
//   g = dy w,  xh = (x - mean) rstd
//   dx = rstd (g - mean(g) - xh mean(g xh)),  dw = sum dy xh,  db = sum dy
//
// Bound by memory: a row is read once into registers, its sums are taken there
// (the variance about the mean), and its results are written.  All sums are fp32.
// Forward, on pairs of fp32: 32768 x 1024 fp32 -> bf16 37 us (31 at the rate of a plain
// copy), 262144 x 128 bf16 26 us (21; on single fp32 33: bound by the issue slots then).
//
// A row is held by `tpr` threads, thread l with the groups l, l + tpr, ... of VEC
// elements: lanes of a warp (tpr <= 32, 32 / tpr rows a warp), or a whole CTA.
// VEC = 8 moves 16 bytes at a time and needs 16-byte rows; VEC = 1 takes any size
// and alignment.
//
// Backward: CTAs stay and take rows in turn; a thread adds up dw and db of its own
// columns in registers over all its rows, the CTA writes one partial sum per
// column, and a second kernel joins the CTAs' sums in a fixed order (the same bits
// every call).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pararnn_sm100.cuh"

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
  int D, nparts, tpr;
  float eps;
};

constexpr int kNormThreads = 256;  // of a CTA whose warps hold whole rows

template <int VEC> __device__ __forceinline__ void norm_load(const float* p, float* v) {
  if constexpr (VEC == 8) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = __ldcs(p);
  }
}
template <int VEC> __device__ __forceinline__ void norm_load(const __nv_bfloat16* p, float* v) {
  if constexpr (VEC == 8) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    const unsigned u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
    v[0] = __bfloat162float(*p);
  }
}
// weights: read again by every row, so they stay in the caches
template <int VEC> __device__ __forceinline__ void norm_weight(const float* p, int at, float none,
                                                               float* v) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = none;
  if (!p) return;
  if constexpr (VEC == 8) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + at));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p + at) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = __ldg(p + at);
  }
}
template <int VEC> __device__ __forceinline__ void norm_store(float* p, const float* v) {
  if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}
template <int VEC> __device__ __forceinline__ void norm_store(__nv_bfloat16* p, const float* v) {
  if constexpr (VEC == 8) {
    unsigned u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const unsigned*>(&t);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    *p = __float2bfloat16_rn(v[0]);
  }
}

// Sums of N values over a row's threads, in every one of them.  In a CTA the
// shared array is used in turns (turn = 0, 1, 0, ...), so one barrier does.
template <int N, bool CTA>
__device__ __forceinline__ void norm_sum(float* v, int tpr, float (*sm)[2][N], int turn) {
  const int width = CTA ? 32 : tpr;
  for (int s = width >> 1; s > 0; s >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], s);
  }
  if constexpr (CTA) {
    const int warp = threadIdx.x >> 5, nw = tpr >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) sm[warp][turn][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int w = 0; w < nw; ++w) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += sm[w][turn][i];
    }
  }
}

// A group's elements as the arithmetic takes them: four pairs, or one number.
template <int VEC> struct NormVal;
template <> struct NormVal<8> {
  using T = f32x2;
  static constexpr int N = 4;
};
template <> struct NormVal<1> {
  using T = float;
  static constexpr int N = 1;
};
__device__ __forceinline__ float nadd(float a, float b) { return a + b; }
__device__ __forceinline__ float nmul(float a, float b) { return a * b; }
__device__ __forceinline__ float nfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ f32x2 nadd(f32x2 a, f32x2 b) { return add2(a, b); }
__device__ __forceinline__ f32x2 nmul(f32x2 a, f32x2 b) { return mul2(a, b); }
__device__ __forceinline__ f32x2 nfma(f32x2 a, f32x2 b, f32x2 c) { return fma2(a, b, c); }
__device__ __forceinline__ void nset(float& d, float v) { d = v; }
__device__ __forceinline__ void nset(f32x2& d, float v) { d = pair2(v, v); }
__device__ __forceinline__ float nsum(float v) { return v; }
__device__ __forceinline__ float nsum(f32x2 v) {
  float x, y;
  unpair2(v, x, y);
  return x + y;
}
__device__ __forceinline__ void nget(const float* v, float* out) { out[0] = v[0]; }
__device__ __forceinline__ void nget(const f32x2* v, float* out) {
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair2(v[i], out[2 * i], out[2 * i + 1]);
}
__device__ __forceinline__ void nput(const float* in, float* v) { v[0] = in[0]; }
__device__ __forceinline__ void nput(const float* in, f32x2* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pair2(in[2 * i], in[2 * i + 1]);
}

// A group as it lies in memory.
template <typename T, int VEC> struct NormRaw;
template <> struct NormRaw<float, 8> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void get(f32x2* v) const {
    v[0] = pair2(a.x, a.y), v[1] = pair2(a.z, a.w);
    v[2] = pair2(b.x, b.y), v[3] = pair2(b.z, b.w);
  }
};
template <> struct NormRaw<__nv_bfloat16, 8> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(f32x2* v) const {
    const unsigned u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pair2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  }
};
template <typename T> struct NormRaw<T, 1> {
  float a;
  __device__ __forceinline__ void load(const T* p) { norm_load<1>(p, &a); }
  __device__ __forceinline__ void zero() { a = 0.0f; }
  __device__ __forceinline__ void get(float* v) const { v[0] = a; }
};

template <typename TX, typename TY, int VEC, int G, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kNormThreads)
    pararnn_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sm[CTA ? 16 : 1][2][1];
  const int lane = threadIdx.x & 31;
  const int l = CTA ? (int)threadIdx.x : lane % p.tpr;
  const long long row = CTA ? (long long)blockIdx.x
                            : (blockIdx.x * (long long)(kNormThreads / 32) + (threadIdx.x >> 5)) *
                                      (32 / p.tpr) + lane / p.tpr;
  const bool live = row < p.M;  // the same for every thread of a row
  const int ng = p.D / VEC;
  const TX* x = static_cast<const TX*>(p.x) + row * p.sx;
  using V = NormVal<VEC>;
  using T = typename V::T;
  constexpr int N = V::N;
  T v[G][N], sum;
  float s[1];
  nset(sum, 0.0f);
  NormRaw<TX, VEC> raw[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int at = l + g * p.tpr;
    raw[g].zero();
    if (live && at < ng) raw[g].load(x + at * VEC);
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    raw[g].get(v[g]);
#pragma unroll
    for (int i = 0; i < N; ++i) sum = nadd(sum, v[g][i]);
  }
  s[0] = nsum(sum);
  norm_sum<1, CTA>(s, p.tpr, sm, 0);
  const float mean = s[0] / (float)p.D;
  T minus;
  nset(minus, -mean);
  nset(sum, 0.0f);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (l + g * p.tpr < ng) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[g][i] = nadd(v[g][i], minus);
        sum = nfma(v[g][i], v[g][i], sum);
      }
    }
  }
  s[0] = nsum(sum);
  norm_sum<1, CTA>(s, p.tpr, sm, 1);
  const float rstd = 1.0f / sqrtf(s[0] / (float)p.D + p.eps);
  if (!live) return;
  TY* y = static_cast<TY*>(p.y) + row * p.D;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int at = (l + g * p.tpr) * VEC;
    if (at < p.D) {
      float w[VEC], b[VEC], out[VEC];
      T w2[N], b2[N], rs;
      norm_weight<VEC>(p.w, at, 1.0f, w);
      norm_weight<VEC>(p.b, at, 0.0f, b);
      nput(w, w2);
      nput(b, b2);
      nset(rs, rstd);
#pragma unroll
      for (int i = 0; i < N; ++i) v[g][i] = nfma(nmul(v[g][i], rs), w2[i], b2[i]);
      nget(v[g], out);
      norm_store<VEC>(y + at, out);
    }
  }
  if (l == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
}

// R rows at a time, and the next R on their way while these are worked on: what is in
// flight covers the latency of HBM.  The rows stay as they lie in memory and are
// unpacked twice (for the sums, and for dx), which costs fewer registers than keeping
// them as fp32.  Measured on B200 (both kernels, us, floor in brackets): 262144 x 128
// bf16 44 (31), 32768 x 1024 fp32 x, bf16 dy 63 (51), 16384 x 4096 the same types 121
// (103).  Bound by the loads in flight (16 warps of 128 registers a SM), at 128 columns by
// the issue slots too: single fp32 operations took 45 / 64 / 127.  Not kept: R = 1 at three
// CTAs a SM 46 / 72 / 137; R = 4 spills, 70 / 105 / 232; two groups of 8 a thread 49 / 78 /
// 144 when one took 48 / 67 / 129; the rows on their way in shared memory (four stages
// of cp.async, each thread its own) 45 / 82 / 178.
template <typename TX, typename TY, int VEC, int G, int R, bool CTA>
__global__ void __launch_bounds__(CTA ? 512 : kNormThreads, CTA ? 1 : 2)
    pararnn_norm_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sm[CTA ? 16 : 1][2][2 * R];
  extern __shared__ float cols[];  // without CTA: [2][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = CTA ? (int)threadIdx.x : lane % p.tpr;
  const int rpw = CTA ? 1 : 32 / p.tpr;                  // rows side by side in a warp
  const int rpc = CTA ? 1 : rpw * (kNormThreads / 32);   // and in a CTA
  const long long stride = (long long)gridDim.x * rpc;   // from one row of a thread to the next
  const int ng = p.D / VEC;
  const float inv = 1.0f / (float)p.D;
  using V = NormVal<VEC>;
  using T = typename V::T;
  constexpr int N = V::N;
  constexpr bool KEEP = G * VEC <= 16;  // the weights stay in registers
  T aw[G][N], ab[G][N], w[KEEP ? G : 1][N];
  const auto weight = [&](int at, T* out) {
    float v[VEC];
    norm_weight<VEC>(at < ng ? p.w : nullptr, at * VEC, 1.0f, v);
    nput(v, out);
  };
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if constexpr (KEEP) weight(l + g * p.tpr, w[g]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      nset(aw[g][i], 0.0f);
      nset(ab[g][i], 0.0f);
    }
  }
  struct Rows {
    NormRaw<TX, VEC> x[R][G];
    NormRaw<TY, VEC> dy[R][G];
    float mean[R], rstd[R];
  };
  const auto fetch = [&](Rows& q, long long row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = row0 + r * stride;
      const bool live = row < p.M;
      q.mean[r] = live ? __ldg(p.mean + row) : 0.0f;
      q.rstd[r] = live ? __ldg(p.rstd + row) : 0.0f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int at = l + g * p.tpr;
        q.x[r][g].zero();
        q.dy[r][g].zero();
        if (live && at < ng) {
          q.x[r][g].load(static_cast<const TX*>(p.x) + row * p.sx + at * VEC);
          q.dy[r][g].load(static_cast<const TY*>(p.dy) + row * p.sdy + at * VEC);
        }
      }
    }
  };
  const long long lead = blockIdx.x * (long long)rpc + (CTA ? 0 : warp * rpw);  // uniform in a warp
  const long long own = CTA ? 0 : lane / p.tpr;
  const auto work = [&](const Rows& cur, long long row0, int turn) {
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      T sg, sgx, minus, rs;
      nset(sg, 0.0f);
      nset(sgx, 0.0f);
      nset(minus, -cur.mean[r]);
      nset(rs, cur.rstd[r]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        T x[N], dy[N], wr[N];
        cur.x[r][g].get(x);
        cur.dy[r][g].get(dy);
        if constexpr (!KEEP) weight(l + g * p.tpr, wr);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const T xh = nmul(nadd(x[i], minus), rs);
          const T dyw = nmul(dy[i], KEEP ? w[KEEP ? g : 0][i] : wr[i]);
          aw[g][i] = nfma(dy[i], xh, aw[g][i]);
          ab[g][i] = nadd(ab[g][i], dy[i]);
          sg = nadd(sg, dyw);
          sgx = nfma(dyw, xh, sgx);
        }
      }
      s[2 * r] = nsum(sg);
      s[2 * r + 1] = nsum(sgx);
    }
    norm_sum<2 * R, CTA>(s, p.tpr, sm, turn);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long long row = row0 + r * stride;
      if (row < p.M) {
        T mg, mgx, minus, rs;  // the means negated
        nset(mg, -s[2 * r] * inv);
        nset(mgx, -s[2 * r + 1] * inv);
        nset(minus, -cur.mean[r]);
        nset(rs, cur.rstd[r]);
        TX* dx = static_cast<TX*>(p.y) + row * p.D;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int at = l + g * p.tpr;
          if (at < ng) {
            T x[N], dy[N], wr[N];
            cur.x[r][g].get(x);
            cur.dy[r][g].get(dy);
            if constexpr (!KEEP) weight(at, wr);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const T xh = nmul(nadd(x[i], minus), rs);
              const T dyw = nmul(dy[i], KEEP ? w[KEEP ? g : 0][i] : wr[i]);
              x[i] = nmul(rs, nfma(xh, mgx, nadd(dyw, mg)));
            }
            float out[VEC];
            nget(x, out);
            norm_store<VEC>(dx + at * VEC, out);
          }
        }
      }
    }
  };
  const long long step = R * stride;
  if constexpr (G * VEC <= 16) {
    Rows one, two;
    int turn = 0;
    fetch(one, lead + own);
    for (long long r0 = lead; r0 < p.M; r0 += step, turn ^= 1) {
      fetch(two, r0 + own + step);
      work(one, r0 + own, turn);
      one = two;
    }
  } else {  // four groups a thread leave no room for a second set
    Rows one;
    int turn = 0;
    for (long long r0 = lead; r0 < p.M; r0 += step, turn ^= 1) {
      fetch(one, r0 + own);
      work(one, r0 + own, turn);
    }
  }

  // one partial sum per column and CTA
  float* pw = p.nparts > 1 ? p.part + (long long)blockIdx.x * p.D : p.dw;
  float* pb = p.nparts > 1 ? p.part + (long long)(p.nparts + blockIdx.x) * p.D : p.db;
  float sw[G][VEC], sb[G][VEC];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    nget(aw[g], sw[g]);
    nget(ab[g], sb[g]);
  }
  if constexpr (!CTA) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        for (int t = p.tpr; t < 32; t <<= 1) {
          sw[g][i] += __shfl_xor_sync(0xffffffffu, sw[g][i], t);
          sb[g][i] += __shfl_xor_sync(0xffffffffu, sb[g][i], t);
        }
    }
    for (int w = 0; w < kNormThreads / 32; ++w) {  // the warps in turn
      if (warp == w && lane < p.tpr) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int at = (l + g * p.tpr) * VEC;
          if (at < p.D) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              cols[at + i] = (w ? cols[at + i] : 0.0f) + sw[g][i];
              cols[p.D + at + i] = (w ? cols[p.D + at + i] : 0.0f) + sb[g][i];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int d = threadIdx.x; d < p.D; d += kNormThreads) {
      pw[d] = cols[d];
      pb[d] = cols[p.D + d];
    }
  } else {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int at = (l + g * p.tpr) * VEC;
      if (at < p.D) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          pw[at + i] = sw[g][i];
          pb[at + i] = sb[g][i];
        }
      }
    }
  }
}

// The CTAs' sums, joined in a fixed order: 32 columns x 32 slices of the parts, a
// slice's loads all in flight (with 8 slices in turn this took 31 us at D = 128,
// as long as the pass itself).
constexpr int kNormSlices = 32;
__global__ void __launch_bounds__(32 * kNormSlices)
    pararnn_norm_join_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sm[kNormSlices][2][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, d = blockIdx.x * 32 + lane;
  float sw = 0.0f, sb = 0.0f;
  wait_for_launch_before();
  if (d < p.D) {
    for (int i0 = slice; i0 < p.nparts; i0 += 8 * kNormSlices) {
      float w[8], b[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * kNormSlices;
        w[k] = i < p.nparts ? __ldcg(p.part + (long long)i * p.D + d) : 0.0f;
        b[k] = i < p.nparts ? __ldcg(p.part + (long long)(p.nparts + i) * p.D + d) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        sw += w[k];
        sb += b[k];
      }
    }
  }
  sm[slice][0][lane] = sw;
  sm[slice][1][lane] = sb;
  __syncthreads();
  if (slice < 2 && d < p.D) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormSlices; ++i) s += sm[i][slice][lane];
    (slice ? p.db : p.dw)[d] = s;
  }
}

// ---- rows of any length (longer than the threads' registers hold) -------------------
__device__ __forceinline__ float norm_block_sum(float v, float* sm) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) v += sm[w];
  return v;
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(1024)
    pararnn_norm_long_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sm[32];
  const long long row = blockIdx.x;
  const TX* x = static_cast<const TX*>(p.x) + row * p.sx;
  TY* y = static_cast<TY*>(p.y) + row * p.D;
  float s = 0.0f, v[1], w[1], b[1];
  for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
    norm_load<1>(x + d, v);
    s += v[0];
  }
  const float mean = norm_block_sum(s, sm) / (float)p.D;
  s = 0.0f;
  for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
    norm_load<1>(x + d, v);
    s = fmaf(v[0] - mean, v[0] - mean, s);
  }
  const float rstd = 1.0f / sqrtf(norm_block_sum(s, sm) / (float)p.D + p.eps);
  for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
    norm_load<1>(x + d, v);
    norm_weight<1>(p.w, d, 1.0f, w);
    norm_weight<1>(p.b, d, 0.0f, b);
    v[0] = fmaf((v[0] - mean) * rstd, w[0], b[0]);
    norm_store<1>(y + d, v);
  }
  if (threadIdx.x == 0) {
    p.mean[row] = mean;
    p.rstd[row] = rstd;
  }
}

template <typename TX, typename TY>
__global__ void __launch_bounds__(1024)
    pararnn_norm_long_dx_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sm[32];
  const long long row = blockIdx.x;
  const TX* x = static_cast<const TX*>(p.x) + row * p.sx;
  const TY* dy = static_cast<const TY*>(p.dy) + row * p.sdy;
  TX* dx = static_cast<TX*>(p.y) + row * p.D;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float sg = 0.0f, sgx = 0.0f, v[1], g[1], w[1];
  for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
    norm_load<1>(x + d, v);
    norm_load<1>(dy + d, g);
    norm_weight<1>(p.w, d, 1.0f, w);
    sg += g[0] * w[0];
    sgx = fmaf(g[0] * w[0], (v[0] - mean) * rstd, sgx);
  }
  const float mg = norm_block_sum(sg, sm) / (float)p.D;
  const float mgx = norm_block_sum(sgx, sm) / (float)p.D;
  for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
    norm_load<1>(x + d, v);
    norm_load<1>(dy + d, g);
    norm_weight<1>(p.w, d, 1.0f, w);
    v[0] = rstd * (g[0] * w[0] - mg - (v[0] - mean) * rstd * mgx);
    norm_store<1>(dx + d, v);
  }
}

// column sums of one slice of rows: thread = column
template <typename TX, typename TY>
__global__ void __launch_bounds__(128)
    pararnn_norm_long_dw_kernel(const __grid_constant__ NormParams p) {
  const int d = blockIdx.x * 128 + threadIdx.x;
  if (d >= p.D) return;
  const long long lo = p.M * blockIdx.y / p.nparts, hi = p.M * (blockIdx.y + 1) / p.nparts;
  float sw = 0.0f, sb = 0.0f, v[1], g[1];
  for (long long r = lo; r < hi; ++r) {
    norm_load<1>(static_cast<const TY*>(p.dy) + r * p.sdy + d, g);
    norm_load<1>(static_cast<const TX*>(p.x) + r * p.sx + d, v);
    sw = fmaf(g[0], (v[0] - p.mean[r]) * p.rstd[r], sw);
    sb += g[0];
  }
  if (p.nparts > 1) {
    p.part[(long long)blockIdx.y * p.D + d] = sw;
    p.part[(long long)(p.nparts + blockIdx.y) * p.D + d] = sb;
  } else {  // one slice: its sums are the result, and there is no workspace
    p.dw[d] = sw;
    p.db[d] = sb;
  }
}

}  // namespace pararnn
