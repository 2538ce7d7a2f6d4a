// pararnn_linattn.cuh -- linear attention with one decay per head: the affine
// scan whose state is a Dk x Dv matrix per (batch row, head).
//
//   S_t = gamma S_{t-1} + k_t^T v_t,   o_t = q_t S_t,   gamma = exp(log_decay[h])
//
// Every kernel here computes one "pass": a walk over time that reads three
// streams (q, k, v roles), carries the state and writes one output stream.
// The forward scan is one such pass; the gradients are three:
//   dq = pass(q: do, k: v, v: k),  forwards, state S^T
//   dk = pass(q: v, k: do, v: q),  backwards, state dS^T
//   dv = pass(q: k, k: q, v: do),  backwards, state dS
// Going backwards the carried state is D = dl/dS_{t-1}: at token t
//   R = D + c_kv k_t^T v_t,  o_t = c_out q_t R,  D <- gamma R,
// and going forwards
//   S <- gamma S + c_kv k_t^T v_t,  o_t = c_out q_t S.
// c_out and c_kv place the attention scale where it belongs in each pass.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pararnn_sm100.cuh"

namespace pararnn {

constexpr int kLaMaxDim = 128;   // largest Dk and Dv
constexpr int kLaMaxPasses = 3;

// One input stream [B, L, Hx, D]: element strides, and the number of heads of
// the pass that share one head of the stream.
struct LaIn {
  const void* p;
  long long sb, st, sh;
  int rep;
};

struct LaPass {
  LaIn q, k, v;
  void* o;               // [B, L, H, dv]: bf16, or fp32 where o_f32
  long long ob, ot, oh;  // element strides of o
  const float* s_in;     // initial state or NULL (= 0): element (r, c) of (b, h) at
  float* s_out;          //   ((b H + h) dk dv) + r s_r + c s_c;  final state or NULL
  long long s_r, s_c;    // the strides of s_in
  float* s_span;         // the spans' states, [B, H, spans, dk, dv]
  int dk, dv;            // contraction and output sizes of this pass
  int rev;               // 1: backwards in time
  int o_f32;
  float c_out, c_kv;
};

struct LaParams {
  LaPass pass[kLaMaxPasses];
  int npass;
  const float* log_decay;  // [H]
  const int* lengths;      // [B] or NULL (= L)
  int B, H;
  long long L;
  int zero_tail;           // write zeros to output rows at and after the length
  int* status_dev;         // 0 / 4, or NULL
  long long timeout_ns;    // bound of the chunked form's waits
  int nspan;               // spans of time, walked side by side
  long long span;          // tokens of a span
};

__device__ __forceinline__ float la_load(const float* p) { return *p; }
__device__ __forceinline__ float la_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ long long la_length(const LaParams& p, int b) {
  if (!p.lengths) return p.L;
  const long long n = p.lengths[b];
  return n < 0 ? 0 : (n > p.L ? p.L : n);
}

// Tokens of span g of batch row b (one span: the whole row).
__device__ __forceinline__ long long la_span_tokens(const LaParams& p, int b, int g) {
  const long long n = la_length(p, b) - g * p.span;
  return n < 0 ? 0 : (p.nspan > 1 && n > p.span ? p.span : n);
}

// gamma^i in 64 bits; gamma^0 = 1 also for gamma = 0
__device__ __noinline__ inline double la_powl(float log_decay, long long i) {
  return i == 0 ? 1.0 : exp((double)log_decay * (double)i);
}
__device__ __forceinline__ double la_pow(float log_decay, int i) { return la_powl(log_decay, i); }

// gamma^i = hi + lo, i > 0, with hi rounded towards zero.  Where gamma is not zero neither hi
// nor lo is, and neither is negative: hi x + lo x keeps an infinite x as the recurrence does
// (0 inf or inf - inf would be NaN).  The least value, 2^-149, is far below every rounding of a
// normal hi; a smaller gamma^i becomes twice that.
constexpr float kLaLeast = 1.40129846e-45f;
__device__ __noinline__ inline float2 la_two(float log_decay, long long i) {
  const double x = exp((double)log_decay * (double)i);
  float hi = __double2float_rz(x), lo = (float)(x - (double)hi);
  if (log_decay > -INFINITY) {
    hi = fmaxf(hi, kLaLeast);
    lo = fmaxf(lo, kLaLeast);
  }
  return make_float2(hi, lo);
}
__device__ __forceinline__ void la_two(float log_decay, long long i, float& hi, float& lo) {
  const float2 two = la_two(log_decay, i);
  hi = two.x;
  lo = two.y;
}

// ---------------------------------------------------------------------------
// Recurrent form.  THREADS threads hold a COLS-column tile of one (b, h) state in
// registers (float4 across, the rest row groups, at most 4 rows a thread) and
// walk the tokens, kLaRecT at a time: the tokens' q, k and v are staged in shared
// memory as fp32, every thread updates its rows and adds up its part of q S, and
// the row groups' parts are joined once per batch of tokens.  All arithmetic is
// fp32.
// ---------------------------------------------------------------------------
constexpr int kLaRecT = 8;
constexpr int kLaRecCols = 32;
constexpr int kLaRecThreads = 256;

template <int COLS> struct LaWalkSmem {
  float q[kLaRecT][kLaMaxDim], k[kLaRecT][kLaMaxDim];
  float v[kLaRecT][COLS];
  float part[kLaRecT][16][COLS];  // one row per warp
};

// Tokens [tb, tb + n) of (b, h), columns c0 .. c0 + COLS - 1, state at element
// (r, c) of s_in + r sr + c sc (NULL = 0); the state behind them to s_out (dense).
template <int COLS, int THREADS>
__device__ __noinline__ void la_walk(const LaParams& p, const LaPass& a, int b, int h, int c0,
                                     long long tb, long long n, const float* s_in, long long sr,
                                     long long sc, float* s_out, LaWalkSmem<COLS>& sm) {
  constexpr int CG = COLS / 4;          // threads across
  constexpr int RG = THREADS / CG;      // row groups: rows rg, rg + RG, ...
  constexpr int R = kLaMaxDim / RG;     // rows a thread
  constexpr int NW = THREADS / 32;
  static_assert(R * RG == kLaMaxDim && NW <= 16 && CG <= 16, "tile");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cg = tid % CG, rg = tid / CG;
  const int col = c0 + cg * 4;  // dv is a multiple of 8: a group of 4 is whole
  const bool cok = col < a.dv;
  const auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory"); };
  // gamma as a sum of two floats: a slow head's memory multiplies by it thousands
  // of times, and the half step that one float leaves (2^-25 near 1) would add up
  // in the same direction every time
  float gamma, glow;
  la_two(p.log_decay[h], 1, gamma, glow);

  float s[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = r * RG + rg;
#pragma unroll
    for (int c = 0; c < 4; ++c) s[r][c] = 0.0f;
    if (s_in && cok && row < a.dk) {
      const float* sp = s_in + row * sr + col * sc;
      if (sc == 1) {
        const float4 x = *reinterpret_cast<const float4*>(sp);
        s[r][0] = x.x, s[r][1] = x.y, s[r][2] = x.z, s[r][3] = x.w;
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[r][c] = sp[c * sc];
      }
    }
  }

  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q.p) + b * a.q.sb + (h / a.q.rep) * a.q.sh;
  const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k.p) + b * a.k.sb + (h / a.k.rep) * a.k.sh;
  const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v.p) + b * a.v.sb + (h / a.v.rep) * a.v.sh;
  const long long obase = b * a.ob + h * a.oh;
  const long long first = a.rev ? tb + n - 1 : tb;
  const int dir = a.rev ? -1 : 1;

  for (long long i0 = 0; i0 < n; i0 += kLaRecT) {
    const int m = (int)(n - i0 < kLaRecT ? n - i0 : kLaRecT);
    sync();  // the staged tokens and parts of the batch before have been read
    for (int e = tid; e < m * a.dk; e += THREADS) {
      const int j = e / a.dk, d = e % a.dk;
      const long long t = first + dir * (i0 + j);
      sm.q[j][d] = la_load(q + t * a.q.st + d);
      sm.k[j][d] = la_load(k + t * a.k.st + d);
    }
    for (int e = tid; e < m * COLS; e += THREADS) {
      const int j = e / COLS, d = e % COLS;
      const long long t = first + dir * (i0 + j);
      sm.v[j][d] = c0 + d < a.dv ? a.c_kv * la_load(v + t * a.v.st + c0 + d) : 0.0f;
    }
    sync();
    for (int j = 0; j < m; ++j) {
      float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      float x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = sm.v[j][cg * 4 + c];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int row = r * RG + rg;
        if (row < a.dk) {
          const float kk = sm.k[j][row], qq = sm.q[j][row];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float old = s[r][c];
            const float w = fmaf(kk, x[c], a.rev ? old : fmaf(gamma, old, glow * old));
            o[c] = fmaf(qq, w, o[c]);
            s[r][c] = a.rev ? fmaf(gamma, w, glow * w) : w;
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int g = CG; g < 32; g <<= 1) o[c] += __shfl_xor_sync(0xffffffffu, o[c], g);
        if (lane < CG) sm.part[j][warp][cg * 4 + c] = o[c];
      }
    }
    sync();
    for (int e = tid; e < m * COLS; e += THREADS) {
      const int j = e / COLS, d = e % COLS;
      if (c0 + d < a.dv) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) x += sm.part[j][w][d];
        x *= a.c_out;
        const long long at = obase + (first + dir * (i0 + j)) * a.ot + c0 + d;
        if (a.o_f32)
          static_cast<float*>(a.o)[at] = x;
        else
          static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(x);
      }
    }
  }

  if (s_out && cok) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = r * RG + rg;
      if (row < a.dk)
        *reinterpret_cast<float4*>(s_out + (long long)row * a.dv + col) =
            make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
    }
  }
}

__global__ void __launch_bounds__(kLaRecThreads)
    pararnn_linattn_recurrent_kernel(const __grid_constant__ LaParams p) {
  __shared__ LaWalkSmem<kLaRecCols> sm;
  const LaPass& a = p.pass[blockIdx.z];
  const int c0 = blockIdx.y * kLaRecCols;
  if (c0 >= a.dv) return;
  const int b = (int)(blockIdx.x / p.H), h = (int)(blockIdx.x % p.H);
  const long long n = la_length(p, b);
  const long long sb = ((long long)b * p.H + h) * a.dk * a.dv;
  la_walk<kLaRecCols, kLaRecThreads>(p, a, b, h, c0, 0, n, a.s_in ? a.s_in + sb : nullptr, a.s_r,
                                        a.s_c, a.s_out ? a.s_out + sb : nullptr, sm);
  if (p.zero_tail) {
    const int warp = threadIdx.x >> 5, d = c0 + (threadIdx.x & 31);
    for (long long t = n + warp; t < p.L; t += kLaRecThreads / 32)
      if (d < a.dv) {
        const long long at = b * a.ob + h * a.oh + t * a.ot + d;
        if (a.o_f32)
          static_cast<float*>(a.o)[at] = 0.0f;
        else
          static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(0.0f);
      }
  }
}

// One token (the decode step): s_next = gamma s + k^T v, o = c_out q s_next.  Bound by
// the state's traffic, 8 dk dv bytes per (b, h).  A CTA has a tile of COLS columns of
// the state of one (b, h): COLS / 4 lanes x float4 across, the rest down, R rows a
// thread, all of whose loads are issued before anything is waited for; the small
// vectors come straight from global memory.  In place is fine: each element is read
// and written by the same thread.  Measured on B200 at 192 x 32 states of 128 x 128 (the
// floor is 124 us): tiles of 32 columns on pairs of fp32 130 us; on single ones 155, and
// 143 with gamma as one float; whole rows of 128 (16 rows a thread, as the 143) 158.
constexpr int kLaStepThreads = 256;

// PART: fewer than ROWS rows, each asked for.  With those conditions where all rows are there
// 256 x 32 states of 64 x 64 take 49 us, without 45; 192 x 32 of 96 x 96 take 93 either way.
// Six CTAs a SM (40 registers; five that take 48: 131 and 47 us at 128 and 64).
template <typename T, int COLS, int ROWS, bool PART>
__global__ void __launch_bounds__(kLaStepThreads, 6)
    pararnn_linattn_step_kernel(const __grid_constant__ LaParams p) {
  constexpr int CG = COLS / 4, RG = kLaStepThreads / CG, R = ROWS / RG;
  __shared__ float4 s_part[kLaStepThreads / 32][CG];
  const LaPass& a = p.pass[0];
  const int tiles = (a.dv + COLS - 1) / COLS;
  const int bh = (int)(blockIdx.x / tiles), c0 = (int)(blockIdx.x % tiles) * COLS;
  const int b = bh / p.H, h = bh % p.H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cg = lane % CG, rg = (int)threadIdx.x / CG, col = c0 + cg * 4;
  const bool cok = col < a.dv;
  const long long sb = (long long)bh * a.dk * a.dv;
  ulonglong2 s[R];  // two pairs of neighbouring columns
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = r * RG + rg;
    s[r] = make_ulonglong2(0ull, 0ull);
    if (a.s_in && cok && (!PART || row < a.dk))
      s[r] = __ldcs(reinterpret_cast<const ulonglong2*>(a.s_in + sb + row * a.dv + col));
  }
  const T* q = static_cast<const T*>(a.q.p) + b * a.q.sb + (h / a.q.rep) * a.q.sh;
  const T* k = static_cast<const T*>(a.k.p) + b * a.k.sb + (h / a.k.rep) * a.k.sh;
  const T* v = static_cast<const T*>(a.v.p) + b * a.v.sb + (h / a.v.rep) * a.v.sh;
  f32x2 x0 = 0, x1 = 0;
  if (cok) {
    x0 = pair2(la_load(v + col), la_load(v + col + 1));
    x1 = pair2(la_load(v + col + 2), la_load(v + col + 3));
  }
  float kk[R], qq[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = r * RG + rg;
    kk[r] = !PART || row < a.dk ? la_load(k + row) : 0.0f;
    qq[r] = !PART || row < a.dk ? la_load(q + row) : 0.0f;
  }
  // a slow head's gamma as two floats: the half step that one leaves would add up over its
  // thousands of tokens.  1 + expm1 is off by 2^-23 |1 - gamma| and 2^-49; the first, over the
  // 1 / |1 - gamma| tokens of its memory, is one rounding; a fast head forgets sooner.
  // Both as in la_two: not negative, and zero only for gamma = 0, for infinite states.
  // (exp in 64 bits by one thread and a barrier took 166 us where this took 155)
  const float ld = p.log_decay[h];
  float gamma, glow = 0.0f;
  if (fabsf(ld) < 0.25f) {
    const float less = expm1f(ld);
    gamma = __fadd_rz(1.0f, less);
    glow = less - (gamma - 1.0f);
  } else {
    gamma = expf(ld);
  }
  if (ld > -INFINITY) {
    gamma = fmaxf(gamma, kLaLeast);
    glow = fmaxf(glow, kLaLeast);
  }
  const f32x2 g2 = pair2(gamma, gamma), l2 = pair2(glow, glow);
  f32x2 o0 = 0, o1 = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = r * RG + rg;
    const f32x2 k2 = pair2(kk[r], kk[r]), q2 = pair2(qq[r], qq[r]);
    const f32x2 w0 = fma2(k2, x0, fma2(g2, s[r].x, mul2(l2, s[r].x))),
                w1 = fma2(k2, x1, fma2(g2, s[r].y, mul2(l2, s[r].y)));
    if (!PART || row < a.dk) {  // a row that is not there would make 0 inf of an infinite v
      o0 = fma2(q2, w0, o0);
      o1 = fma2(q2, w1, o1);
      if (cok)
        *reinterpret_cast<ulonglong2*>(a.s_out + sb + row * a.dv + col) = make_ulonglong2(w0, w1);
    }
  }
  float4 o;
  unpair2(o0, o.x, o.y);
  unpair2(o1, o.z, o.w);
#pragma unroll
  for (int m = CG; m < 32; m <<= 1) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
  }
  if (lane < CG) s_part[warp][lane] = o;
  __syncthreads();
  if (threadIdx.x < COLS && c0 + threadIdx.x < a.dv) {
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kLaStepThreads / 32; ++w)
      y += reinterpret_cast<const float*>(s_part[w])[threadIdx.x];
    y *= a.c_out;
    const long long at = b * a.ob + h * a.oh + c0 + threadIdx.x;
    if (a.o_f32)
      static_cast<float*>(a.o)[at] = y;
    else
      static_cast<__nv_bfloat16*>(a.o)[at] = __float2bfloat16_rn(y);
  }
}

// Gradient of a stream whose heads are shared: the fp32 gradients of the H
// heads [rows, H, D] summed in head order over each group -> bf16 [rows, Hx, D].
__global__ void pararnn_linattn_group_kernel(const float* x, __nv_bfloat16* y, long long rows,
                                             int H, int Hx, int D) {
  const int rep = H / Hx, D4 = D / 4;
  const long long n = rows * Hx * D4;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x) {
    const long long rh = i / D4;  // row * Hx + hx
    const int d = (int)(i % D4) * 4;
    const float* s = x + (rh * rep) * D + d;
    float4 acc = *reinterpret_cast<const float4*>(s);
    for (int g = 1; g < rep; ++g) {
      const float4 w = *reinterpret_cast<const float4*>(s + (long long)g * D);
      acc.x += w.x, acc.y += w.y, acc.z += w.z, acc.w += w.w;
    }
    __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(y + rh * D + d);
    out[0] = __floats2bfloat162_rn(acc.x, acc.y);
    out[1] = __floats2bfloat162_rn(acc.z, acc.w);
  }
}

}  // namespace pararnn
