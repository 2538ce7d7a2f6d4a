// pararnn_linattn_chunk.cuh -- linear attention by chunks of 128 tokens on the
// tensor cores (tcgen05, bf16 operands, fp32 accumulation).
//
// Within a chunk of n tokens with the state S at its start (forwards):
//   o_i  = c_out (gamma^(i+1) q_i S + c_kv sum_{j<=i} gamma^(i-j) (q_i.k_j) v_j)
//   S'   = gamma^n S + sum_j k_j^T (c_kv gamma^(n-1-j) v_j)
// and backwards in time, with D = dl/dS after the chunk:
//   o_i  = c_out (gamma^(n-1-i) q_i D + c_kv sum_{j>=i} gamma^(j-i) (q_i.k_j) v_j)
//   D'   = gamma^n D + sum_j k_j^T (c_kv gamma^(j+1) v_j)
//
// One CTA walks the chunks of one (batch row, head) and one 64-column tile of
// the state, which stays in registers (fp32, one state row a thread).  Per chunk
// four products run on the tensor cores:
//   scores  S_qk = Q K^T           128 x 128 x dk    both operands K-major
//   update  U    = K^T [V1 V2 V3]  dk x 192 x 128    both operands MN-major
//   carried O_i  = Q S             128 x 64 x dk
//   local   O_a  = P V             128 x 64 x 128    P from TMEM
// V1 + V2 + V3 are three bf16 pieces of the weighted v (24 bits, so the state
// is as exact as fp32 sums make it); they lie side by side, so that one N = 192
// product reads K^T once for all three.  P (the weighted scores) and the copy of
// S that Q multiplies are rounded to bf16: two independent roundings of terms of
// an output that is itself rounded to bf16.
//
// Roles: warp 0 tensor copies (q, k, v of a chunk, two stages), warp 1 issues
// the products, warps 2-5 weight the scores and write the outputs, warps 6-9
// weight v, carry the state and write its bf16 copy.  Every wait is bounded.
#pragma once

#include "pararnn_linattn.cuh"
#include "pararnn_proj.cuh"

namespace pararnn {

constexpr int kLaT = 128;  // tokens per chunk
constexpr int kLaN = 64;   // state columns per CTA
constexpr int kLaThreads = 320;
constexpr unsigned kLaBlk = kLaT * 128;  // a 128-row block of 64 bf16 columns

template <int KD> struct LaSmem {
  static constexpr unsigned kQ = 0;                                   // [2][KD/64] blocks
  static constexpr unsigned kK = kQ + 2 * (KD / 64) * kLaBlk;         // [2][KD/64] blocks
  static constexpr unsigned kV = kK + 2 * (KD / 64) * kLaBlk;         // [2] blocks
  static constexpr unsigned kVw = kV + 2 * kLaBlk;                    // 3 blocks
  static constexpr unsigned kS = kVw + 3 * kLaBlk;                    // KD rows x 128 B
  static constexpr unsigned kEnd = kS + KD * 128;
  static constexpr size_t kBytes = kEnd + 1024;  // + alignment slack
};

struct LaMaps {
  CUtensorMap q[kLaMaxPasses], k[kLaMaxPasses], v[kLaMaxPasses];
};

// MN-major operand written by tensor copies with the 128-byte swizzle: rows of
// 64 elements along M or N, 8-row groups along K 1024 bytes apart (bits 32-45),
// blocks of 64 along M or N kLaBlk apart (bits 16-29).
__device__ __forceinline__ unsigned long long umma_desc_mn_sw128(unsigned saddr) {
  return (unsigned long long)((saddr & 0x3FFFFu) >> 4) |
         ((unsigned long long)(kLaBlk >> 4) << 16) | ((unsigned long long)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

__host__ __device__ constexpr unsigned la_idesc(unsigned n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | (8u << 24);  // M = 128
}

// A from TMEM (lane = row, two bf16 of K per 32-bit column), B from shared memory.
__device__ __forceinline__ void umma_f16_ts(unsigned tmem_d, unsigned tmem_a,
                                            unsigned long long db, unsigned idesc,
                                            unsigned accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(db), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d_s(unsigned dst, const CUtensorMap* map, int x, int y,
                                              int z, int w, unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(y), "r"(z), "r"(w),
      "r"(smem_u32(bar))
      : "memory");
}

// 32 consecutive columns of this thread's TMEM lane, not waited for.
__device__ __forceinline__ void tmem_ld32_async(unsigned taddr, unsigned* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st16(unsigned taddr, const unsigned* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const unsigned*>(&t);
}
__device__ __forceinline__ float bf16_lo(unsigned u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) { return __uint_as_float(u & 0xFFFF0000u); }

// shared-memory address of the 16-byte unit j of row r of a swizzled block
__device__ __forceinline__ unsigned la_unit(unsigned block, int r, int j) {
  return block + (unsigned)r * 128u + ((unsigned)(j ^ (r & 7)) << 4);
}
__device__ __forceinline__ uint4 lds128(unsigned a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(unsigned a, unsigned x, unsigned y, unsigned z, unsigned w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// x = hi + lo with hi the nearest float (0 beyond the range of a float)
__device__ __forceinline__ void la_two(double x, float& hi, float& lo) {
  hi = (float)x;
  lo = isfinite(hi) ? (float)(x - (double)hi) : 0.0f;
}

// gamma^i in 64 bits; gamma^0 = 1 also for gamma = 0
__device__ __forceinline__ double la_pow(float log_decay, int i) {
  return i == 0 ? 1.0 : exp((double)log_decay * (double)i);
}

template <int KD>
__global__ void __launch_bounds__(kLaThreads, 1)
    pararnn_linattn_chunk_kernel(const __grid_constant__ LaParams p,
                                 const __grid_constant__ LaMaps tm) {
  using Sm = LaSmem<KD>;
  extern __shared__ __align__(1024) unsigned char dsmem[];
  __shared__ unsigned long long s_full[2], s_pv[2], s_sc, s_p, s_kv, s_qs, s_b, s_ofree, s_drain;
  __shared__ __align__(16) float s_pw[kLaT + 4], s_col[32];
  __shared__ unsigned s_tmem;
  __shared__ int s_fail;

  const LaPass& a = p.pass[blockIdx.z];
  const int col0 = blockIdx.y * kLaN;
  if (col0 >= a.dv) return;  // the whole CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = (int)(blockIdx.x / p.H), h = (int)(blockIdx.x % p.H);
  const unsigned sbase = (smem_u32(dsmem) + 1023u) & ~1023u;
  const WaitCtx wctx{nullptr, p.status_dev, p.timeout_ns};
  const long long len = la_length(p, b);
  const int nc = (int)((len + kLaT - 1) / kLaT);
  const float ld = p.log_decay[h];
  const bool rev = a.rev != 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_pv[s], 1);
    }
    mbar_init(&s_sc, 1);
    mbar_init(&s_kv, 1);
    mbar_init(&s_qs, 1);
    mbar_init(&s_drain, 1);
    mbar_init(&s_p, 128);
    mbar_init(&s_b, 128);
    mbar_init(&s_ofree, 128);
    s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&s_tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + kLaT + 1)
    s_pw[threadIdx.x - 64] = (float)la_pow(ld, (int)threadIdx.x - 64);
  if (threadIdx.x < 32)  // the column factor of a 32-column block off the diagonal
    s_col[threadIdx.x] = (float)la_pow(ld, rev ? (int)threadIdx.x : 31 - (int)threadIdx.x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const unsigned tmem = s_tmem;
  const unsigned t_sc = tmem, t_p = tmem + 128, t_kv = tmem + 192, t_oi = tmem + 384,
                 t_oa = tmem + 448;
  // token of row 0 of the c-th chunk walked, and its number of tokens
  const auto t0 = [&](int c) { return (rev ? nc - 1 - c : c) * kLaT; };
  const auto rows = [&](int c) { return (int)(len - t0(c) < kLaT ? len - t0(c) : kLaT); };

  if (warp == 0) {
    if (lane == 0) {
      // ---- tensor copies ----------------------------------------------------------
      const CUtensorMap *mq = &tm.q[blockIdx.z], *mk = &tm.k[blockIdx.z], *mv = &tm.v[blockIdx.z];
      const int hq = h / a.q.rep, hk = h / a.k.rep, hv = h / a.v.rep;
      int c = 0;
      for (; c < nc && !*(volatile int*)&s_fail; ++c) {
        const int st = c & 1;
        // chunk c - 2 is done with this stage
        if (c >= 2 && !stage_wait(&s_pv[st], (unsigned)((c >> 1) - 1) & 1u, wctx)) {
          s_fail = 1;
          break;
        }
        mbar_expect_tx(&s_full[st], (2 * (KD / 64) + 1) * kLaBlk);
        const int t = t0(c);
#pragma unroll
        for (int j = 0; j < KD / 64; ++j) {
          const unsigned off = (st * (KD / 64) + j) * kLaBlk;
          tma_load_4d_s(sbase + Sm::kQ + off, mq, 64 * j, t, hq, b, &s_full[st]);
          tma_load_4d_s(sbase + Sm::kK + off, mk, 64 * j, t, hk, b, &s_full[st]);
        }
        tma_load_4d_s(sbase + Sm::kV + st * kLaBlk, mv, col0, t, hv, b, &s_full[st]);
      }
      // no copy is in flight when the CTA exits (only a failed wait leaves one)
      WaitCtx last = wctx;
      if (last.timeout_ns < 2000000000LL) last.timeout_ns = 2000000000LL;
      for (int i = c - 2 < 0 ? 0 : c - 2; i < c; ++i)
        stage_wait(&s_full[i & 1], (unsigned)(i >> 1) & 1u, last);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---- products ---------------------------------------------------------------
      for (int c = 0; c < nc && !*(volatile int*)&s_fail; ++c) {
        const int st = c & 1;
        const unsigned par = (unsigned)c & 1u;
        const unsigned q = sbase + Sm::kQ + st * (KD / 64) * kLaBlk;
        const unsigned k = sbase + Sm::kK + st * (KD / 64) * kLaBlk;
        const unsigned v = sbase + Sm::kV + st * kLaBlk;
        bool ok = stage_wait(&s_full[st], (unsigned)(c >> 1) & 1u, wctx);
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < KD / 16; ++i) {
            const unsigned off = (i >> 2) * kLaBlk + (i & 3) * 32u;
            umma_f16_ss(t_sc, umma_desc_sw128(q + off), umma_desc_sw128(k + off),
                        la_idesc(128, false, false), i != 0);
          }
          umma_commit(&s_sc);
          ok = stage_wait(&s_b, par, wctx);  // weighted v and the state's copy are there
        }
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < kLaT / 16; ++i)
            umma_f16_ss(t_kv, umma_desc_mn_sw128(k + i * 2048u),
                        umma_desc_mn_sw128(sbase + Sm::kVw + i * 2048u),
                        la_idesc(192, true, true), i != 0);
          umma_commit(&s_kv);
          // the outputs of the chunk before have been read
          if (c > 0) ok = stage_wait(&s_ofree, par ^ 1u, wctx);
        }
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < KD / 16; ++i)
            umma_f16_ss(t_oi, umma_desc_sw128(q + (i >> 2) * kLaBlk + (i & 3) * 32u),
                        umma_desc_mn_sw128(sbase + Sm::kS + i * 2048u),
                        la_idesc(64, false, true), i != 0);
          umma_commit(&s_qs);
          ok = stage_wait(&s_p, par, wctx);
        }
        if (!ok) {
          s_fail = 1;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < kLaT / 16; ++i)
          umma_f16_ts(t_oa, t_p + i * 8, umma_desc_mn_sw128(v + i * 2048u),
                      la_idesc(64, false, true), i != 0);
        umma_commit(&s_pv[st]);
      }
      // every product has completed before the TMEM is given back
      umma_commit(&s_drain);
      WaitCtx last = wctx;
      if (last.timeout_ns < 2000000000LL) last.timeout_ns = 2000000000LL;
      stage_wait(&s_drain, 0u, last);
    }
  } else if (warp < 6) {
    // ---- weighted scores and outputs: thread = token -------------------------------
    const int qd = warp & 3, i = 32 * qd + lane;
    const unsigned lane_off = (unsigned)(32 * qd) << 16;
    const float cs = a.c_out * a.c_kv;
    const long long obase = (long long)b * a.ob + (long long)h * a.oh + col0;
    const int nd = a.dv - col0 < kLaN ? a.dv - col0 : kLaN;
    for (int c = 0; c < nc; ++c) {
      const unsigned par = (unsigned)c & 1u;
      const int n = rows(c);
      bool ok = stage_wait(&s_sc, par, wctx);
      if (!__all_sync(0xffffffffu, ok) || *(volatile int*)&s_fail) {
        s_fail = 1;
        break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int J = 0; J < 4; ++J) {
        unsigned w[16];
        const bool live = rev ? J >= qd : J <= qd;  // uniform in the warp
        if (live) {
          unsigned r[32];
          tmem_ld32_async(t_sc + lane_off + 32 * J, r);
          tmem_wait_ld();
          if (J == qd) {
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x[2];
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const int d = rev ? e + g - lane : lane - e - g;
                const float f = s_pw[d & 127] * cs;
                x[g] = d >= 0 && 32 * J + e + g < n ? __uint_as_float(r[e + g]) * f : 0.0f;
              }
              w[e / 2] = pack_bf16(x[0], x[1]);
            }
          } else {
            const float f = cs * s_pw[rev ? 32 * J - i : i - 32 * J - 31];
            const int m = n - 32 * J;  // columns at and after m are padding
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 cf = *reinterpret_cast<const float4*>(&s_col[e]);
              float x[4] = {__uint_as_float(r[e]) * (f * cf.x),
                            __uint_as_float(r[e + 1]) * (f * cf.y),
                            __uint_as_float(r[e + 2]) * (f * cf.z),
                            __uint_as_float(r[e + 3]) * (f * cf.w)};
              if (m < 32) {
#pragma unroll
                for (int g = 0; g < 4; ++g)
                  if (e + g >= m) x[g] = 0.0f;
              }
              w[e / 2] = pack_bf16(x[0], x[1]);
              w[e / 2 + 1] = pack_bf16(x[2], x[3]);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = 0u;
        }
        tmem_st16(t_p + lane_off + 16 * J, w);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&s_p);

      ok = stage_wait(&s_pv[c & 1], (unsigned)(c >> 1) & 1u, wctx);
      if (!__all_sync(0xffffffffu, ok) || *(volatile int*)&s_fail) {
        s_fail = 1;
        break;
      }
      tc_fence_after();
      const float e = i < n ? a.c_out * s_pw[rev ? n - 1 - i : i + 1] : 0.0f;
      float x[64];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        unsigned y[32], w[32];
        tmem_ld32_async(t_oi + lane_off + 32 * half, y);
        tmem_ld32_async(t_oa + lane_off + 32 * half, w);
        tmem_wait_ld();
#pragma unroll
        for (int d = 0; d < 32; ++d)
          x[32 * half + d] = fmaf(e, __uint_as_float(y[d]), __uint_as_float(w[d]));
      }
      tc_fence_before();
      mbar_arrive(&s_ofree);
      if (i < n) {
        const long long at = obase + (long long)(t0(c) + i) * a.ot;
        if (a.o_f32) {
          float* o = static_cast<float*>(a.o) + at;
#pragma unroll
          for (int d = 0; d < 64; d += 4)
            if (d < nd)
              *reinterpret_cast<float4*>(o + d) = make_float4(x[d], x[d + 1], x[d + 2], x[d + 3]);
        } else {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + at;
#pragma unroll
          for (int d = 0; d < 64; d += 8)
            if (d < nd)
              *reinterpret_cast<uint4*>(o + d) =
                  make_uint4(pack_bf16(x[d], x[d + 1]), pack_bf16(x[d + 2], x[d + 3]),
                             pack_bf16(x[d + 4], x[d + 5]), pack_bf16(x[d + 6], x[d + 7]));
        }
      }
    }
    if (p.zero_tail && !*(volatile int*)&s_fail) {
      for (long long t = len + i; t < p.L; t += kLaT)
        for (int d = 0; d < nd; d += 8) {
          const long long at = obase + t * a.ot + d;
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          if (a.o_f32) {
            *reinterpret_cast<uint4*>(static_cast<float*>(a.o) + at) = zero;
            *reinterpret_cast<uint4*>(static_cast<float*>(a.o) + at + 4) = zero;
          } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + at) = zero;
          }
        }
    }
  } else {
    // ---- weighted v and the state: thread = token, thread = state row --------------
    const int qd = warp & 3, r = 32 * qd + lane;
    const unsigned lane_off = (unsigned)(32 * qd) << 16;
    const bool srow = r < a.dk;
    const long long sb = ((long long)b * p.H + h) * a.dk * a.dv;
    float s[kLaN];
#pragma unroll
    for (int d = 0; d < kLaN; ++d) s[d] = 0.0f;
    if (a.s_in && srow) {
#pragma unroll
      for (int d = 0; d < kLaN; ++d)
        if (col0 + d < a.dv) s[d] = a.s_in[sb + r * a.s_r + (col0 + d) * a.s_c];
    }
    float ghi, glo;  // gamma^128
    la_two(la_pow(ld, kLaT), ghi, glo);
    bool failed = false;
    // s <- gamma^m s + U of the chunk before, which had m tokens
    const auto take = [&](int c) {
      bool ok = stage_wait(&s_kv, (unsigned)c & 1u, wctx);
      if (!__all_sync(0xffffffffu, ok)) return false;
      tc_fence_after();
      float h1 = ghi, h2 = glo;
      const int m = rows(c);
      if (m < kLaT) la_two(la_pow(ld, m), h1, h2);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        unsigned u1[32], u2[32], u3[32];
        tmem_ld32_async(t_kv + lane_off + 32 * half, u1);
        tmem_ld32_async(t_kv + lane_off + 64 + 32 * half, u2);
        tmem_ld32_async(t_kv + lane_off + 128 + 32 * half, u3);
        tmem_wait_ld();
#pragma unroll
        for (int d = 0; d < 32; ++d) {
          const float old = s[32 * half + d];
          const float small = fmaf(h2, old, __uint_as_float(u3[d]) + __uint_as_float(u2[d]));
          s[32 * half + d] = fmaf(h1, old, __uint_as_float(u1[d]) + small);
        }
      }
      return true;
    };
    for (int c = 0; c < nc; ++c) {
      const int st = c & 1, n = rows(c);
      if (c > 0 && !take(c - 1)) {
        failed = true;
        break;
      }
      bool ok = true;
      if (c > 0) ok = stage_wait(&s_qs, (unsigned)(c - 1) & 1u, wctx);  // the copy has been read
      if (ok) ok = stage_wait(&s_full[st], (unsigned)(c >> 1) & 1u, wctx);
      if (!__all_sync(0xffffffffu, ok) || *(volatile int*)&s_fail) {
        failed = true;
        break;
      }
      if (KD == 128 || r < KD) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          sts128(la_unit(sbase + Sm::kS, r, j), pack_bf16(s[8 * j], s[8 * j + 1]),
                 pack_bf16(s[8 * j + 2], s[8 * j + 3]), pack_bf16(s[8 * j + 4], s[8 * j + 5]),
                 pack_bf16(s[8 * j + 6], s[8 * j + 7]));
      }
      const unsigned vb = sbase + Sm::kV + st * kLaBlk, wb = sbase + Sm::kVw;
      const float f = r < n ? a.c_kv * s_pw[rev ? r + 1 : n - 1 - r] : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint4 x = lds128(la_unit(vb, r, j));
        if (r >= n) {  // padding: whatever it holds becomes zero, in k too
          x = make_uint4(0u, 0u, 0u, 0u);
          sts128(la_unit(vb, r, j), 0u, 0u, 0u, 0u);
#pragma unroll
          for (int m = 0; m < KD / 64; ++m)
            sts128(la_unit(sbase + Sm::kK + (st * (KD / 64) + m) * kLaBlk, r, j), 0u, 0u, 0u, 0u);
        }
        const unsigned in[4] = {x.x, x.y, x.z, x.w};
        unsigned w1[4], w2[4], w3[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float y0 = bf16_lo(in[g]) * f, y1 = bf16_hi(in[g]) * f;
          w1[g] = pack_bf16(y0, y1);
          const float z0 = y0 - bf16_lo(w1[g]), z1 = y1 - bf16_hi(w1[g]);
          w2[g] = pack_bf16(z0, z1);
          w3[g] = pack_bf16(z0 - bf16_lo(w2[g]), z1 - bf16_hi(w2[g]));
        }
        sts128(la_unit(wb, r, j), w1[0], w1[1], w1[2], w1[3]);
        sts128(la_unit(wb + kLaBlk, r, j), w2[0], w2[1], w2[2], w2[3]);
        sts128(la_unit(wb + 2 * kLaBlk, r, j), w3[0], w3[1], w3[2], w3[3]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before();
      mbar_arrive(&s_b);
    }
    if (!failed && nc > 0 && !take(nc - 1)) failed = true;
    if (failed) {
      s_fail = 1;
    } else if (a.s_out && srow) {
#pragma unroll
      for (int d = 0; d < kLaN; d += 4)
        if (col0 + d < a.dv)
          *reinterpret_cast<float4*>(a.s_out + sb + (long long)r * a.dv + col0 + d) =
              make_float4(s[d], s[d + 1], s[d + 2], s[d + 3]);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && s_fail && p.status_dev) atomicCAS(p.status_dev, 0, 4);
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

}  // namespace pararnn
