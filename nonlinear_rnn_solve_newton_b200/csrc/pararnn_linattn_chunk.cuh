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
// One CTA walks the chunks of one (batch row, head), one span of time and one
// 64-column tile of the state, which stays in registers (fp32, half a state row a
// thread).  Per chunk four products run on the tensor cores:
//   scores  S_qk = Q K^T           128 x 128 x dk    both operands K-major
//   update  U    = K^T [V1 V2 V3]  dk x 192 x 128    both operands MN-major
//   carried O_i  = Q S             128 x 64 x dk
//   local   O_a  = P V             128 x 64 x 128    P from TMEM
// V1 + V2 + V3 are three bf16 pieces of the weighted v (24 bits, so the state
// is as exact as fp32 sums make it); they lie side by side, so that one N = 192
// product reads K^T once for all three.  A pass whose state nobody gets (dq and dk)
// takes two pieces: the 2^-17 that they leave is far below the bf16 of its output.
// P (the weighted scores) and the copy of
// S that Q multiplies are rounded to bf16: two independent roundings of terms of
// an output that is itself rounded to bf16.
//
// Roles: warp 0 tensor copies (q, k, v of a chunk, two stages each; the output
// tile, staged where the chunk's v was), warp 1 issues the products, warps 2-9
// weight the scores and write the outputs, warps 10-17 carry the state, weight v
// and write the state's bf16 copy.  Two warps share a TMEM lane quarter and split
// its columns: with four warps a role, each instruction was fetched for a single
// warp of an SM quarter and a third of the issue slots waited for instructions.
// Every wait is bounded.
//
// Measured on B200, heads of 128, bf16: 8 x 4096 tokens of 8 heads 75 us (272 MB, 42 us at
// the rate of a plain copy), 8 x 8192 of 32 heads 630-770 us (2.2 GB, 334 us).  A chunk
// takes about 3700 cycles a CTA.  1920 of them are the tensor pipe's (scores 512, update 768,
// carried 384, local 256: 44% in the counters); DRAM is at 36%, the issue slots at 44%.
// What is left is the way of one v buffer: load 1150, weigh 1100, the products, read the
// outputs, stage and store them, load; without any arithmetic of the warps it still takes
// 66 of 79 us.  The largest runs are held by power besides (990 W, the SM clock at 1.35
// to 1.4 of 1.965 GHz), whence the spread.  64 state columns a CTA, not 128: 128 fp32
// states a thread and a third buffer of TMEM do not fit, and half as many CTAs would
// leave SMs idle at 8 x 8 heads.  Not kept (us at 8 x 8192 x 32 heads, same box): outputs
// stored by warps of their own 840 against 787; the first copies issued before the
// rest of the setup 745 against 692; k or v split between the roles: spills.
//
// TMEM (512 columns): two buffers of 128 for the scores -- the weighted scores
// replace the lower half of a buffer, the local output then takes the upper --
// 192 for the update, 64 for the carried output.
//
// A mask that multiplies by zero lets a non-finite k or v of a later token
// of the chunk into an output.  Such a token also leaves the state non-finite
// for good, so the end of the walk shows it.  A product q.k beyond fp32 shows in the
// weighted scores, whose largest is kept (also where v is zero or the token later,
// so that no output should see it).  In both cases the CTA walks its tokens again with
// the recurrent form, which reads no token before its time and makes no scores; in the walk
// of the states only, so that a span leaves the infinities that the recurrence has there.
//
// Spans: where (batch row, head, tile) give fewer CTAs than SMs, time is cut into
// spans.  A first launch (FULL = false) computes the state that each span's own
// tokens leave (54 us of 155 for 65536 tokens of 12 heads of 64, 67 when one role weighted v
// and took the update in turn), pararnn_linattn_join_kernel carries them over the spans, and the
// walk starts each span from the state before it.  In the first launch warps 2-9 weight
// v, into two places in turn, and the update has two buffers, so that weights, product
// and state work on three chunks at a time.
#pragma once

#include "pararnn_linattn.cuh"
#include "pararnn_proj.cuh"
#include "pararnn_sm100.cuh"

namespace pararnn {

constexpr int kLaT = 128;  // tokens per chunk
constexpr int kLaN = 64;   // state columns per CTA
constexpr int kLaWt2 = kLaT + 32 + 16;  // the second copy of the weights
constexpr int kLaThreads = 576;
constexpr int kLaAgainThreads = 512;  // of the recurrent walk over non-finite inputs
// chunks that are brought into L2 ahead of the copies: a buffer is refilled only when
// it falls free, too late for the latency of HBM
constexpr int kLaAhead = 2;
constexpr unsigned kLaBlk = kLaT * 128;  // a 128-row block of 64 bf16 columns

template <int KD> struct LaSmem {
  static constexpr unsigned kQ = 0;                                   // [2][KD/64] blocks
  static constexpr unsigned kK = kQ + 2 * (KD / 64) * kLaBlk;         // [2][KD/64] blocks
  static constexpr unsigned kV = kK + 2 * (KD / 64) * kLaBlk;         // [2] blocks
  static constexpr unsigned kVw = kV + 2 * kLaBlk;                    // 3 blocks
  static constexpr unsigned kS = kVw + 3 * kLaBlk;                    // KD rows x 128 B
  static constexpr unsigned kEnd = kS + KD * 128;
  // a second place for weighted v where no q and no outputs are made (FULL = false)
  static constexpr unsigned kVw2 = KD == 128 ? kQ : kEnd;
  static constexpr size_t bytes(bool full) {  // with alignment slack
    return kEnd + 1024 + (full || KD == 128 ? 0 : 3 * kLaBlk);
  }
};

struct LaMaps {
  CUtensorMap q[kLaMaxPasses], k[kLaMaxPasses], v[kLaMaxPasses], o[kLaMaxPasses];
};

// A wait: one plain try (41 cycles where the phase is over, 90 with a time limit), then
// tries that sleep in the hardware for up to 2 us each, so that the waiting warps leave
// the issue slots to the working ones.
__device__ __forceinline__ bool la_sleep_wait(unsigned long long* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(2000u)
      : "memory");
  return ok != 0u;
}
// the polling loop is a call: twenty copies of it in the roles' loops would crowd them
// out of the instruction caches
__device__ __noinline__ inline bool la_wait_on(unsigned long long* bar, unsigned parity,
                                               long long timeout_ns) {
  const unsigned long long t0 = globaltimer();
  for (;;) {
    if (la_sleep_wait(bar, parity)) return true;
    if (globaltimer() - t0 > (unsigned long long)timeout_ns) return false;
  }
}
__device__ __forceinline__ bool la_wait(unsigned long long* bar, unsigned parity,
                                        long long timeout_ns) {
  return mbar_try_wait(bar, parity) || la_wait_on(bar, parity, timeout_ns);
}

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

// One thread of a converged warp.  The compiler keeps what such a thread uses in uniform
// registers; under `lane == 0` it moves every descriptor there before each
// tcgen05.mma.  Measured on B200, 8 MMAs of M = 128, N = 64 ... 192: 1400-1900
// cycles to issue under lane == 0, 255-750 (the tensor pipe's own time) so.
__device__ __forceinline__ bool la_elect() {
  unsigned p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0u;
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

// 16 consecutive columns of this thread's TMEM lane, not waited for.
__device__ __forceinline__ void tmem_ld16_async(unsigned taddr, unsigned* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
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
// The larger of the magnitudes, in each half; NaN where either is one.
__device__ __forceinline__ unsigned larger_bf16x2(unsigned a, unsigned b) {
  unsigned d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The box on its way into L2 (nothing waits for it).
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<unsigned long long>(map)),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
// A tensor's description on its way into the copies' cache.
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<unsigned long long>(map))
               : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, unsigned src, int x, int y,
                                             int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
          reinterpret_cast<unsigned long long>(map)),
      "r"(x), "r"(y), "r"(z), "r"(w), "r"(src)
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ f32x2 pair2u(unsigned x, unsigned y) {
  return pair2(__uint_as_float(x), __uint_as_float(y));
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

// BWD: a pass of the backward call, whose output may be fp32 and whose state unwanted.
template <int KD, bool FULL, bool BWD>
__global__ void __launch_bounds__(kLaThreads, 1)
    pararnn_linattn_chunk_kernel(const __grid_constant__ LaParams p,
                                 const __grid_constant__ LaMaps tm) {
  using Sm = LaSmem<KD>;
  extern __shared__ __align__(1024) unsigned char dsmem[];
  __shared__ unsigned long long s_full[2], s_vfull[2], s_pv[2], s_put[2], s_sc[2],
      s_rd[4], s_p, s_kv[2], s_qs[2], s_b, s_go[2], s_pad, s_drain;
  // c_out c_kv gamma^d by distance d, in the order in which a row's columns need it:
  // forwards d = 127 - x, backwards d = x - 32; 0 for the 32 distances below 0.  A second
  // copy, one place on and 16 banks off, is for rows whose first place is odd: every
  // row then reads aligned pairs, and no two rows of a half warp the same bank
  __shared__ __align__(16) float s_wt[2 * (kLaT + 32) + 16];
  __shared__ unsigned s_tmem;
  __shared__ int s_fail, s_bad;

  const LaPass& a = p.pass[blockIdx.z];
  const int col0 = blockIdx.y * kLaN;
  if (col0 >= a.dv) return;  // the whole CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = (int)(blockIdx.x / p.nspan), span = (int)(blockIdx.x % p.nspan);
  const int b = bh / p.H, h = bh % p.H;
  const unsigned sbase = (smem_u32(dsmem) + 1023u) & ~1023u;
  const long long limit = p.timeout_ns;
  // the tokens of this CTA: [tb, tb + len)
  const int tb = (int)(span * p.span), len = (int)la_span_tokens(p, b, span);  // L < 2^31
  const int nc = (len + kLaT - 1) / kLaT;
  const float ld = p.log_decay[h];
  const bool rev = a.rev != 0, three = !BWD || a.s_out != nullptr;  // pieces of v
  // the state before this span and behind it: element (r, c) at r s_r + c s_c
  const long long sb = (p.nspan > 1 ? (long long)blockIdx.x : bh) * a.dk * a.dv;
  const float* s_in = !FULL ? nullptr : p.nspan > 1 ? a.s_span : a.s_in;
  float* s_out = !FULL ? a.s_span : p.nspan > 1 ? nullptr : a.s_out;
  const long long sr = p.nspan > 1 ? a.dv : a.s_r, sc = p.nspan > 1 ? 1 : a.s_c;

  if (threadIdx.x == 64) {
    tma_prefetch_map(&tm.k[blockIdx.z]);
    tma_prefetch_map(&tm.v[blockIdx.z]);
    if (FULL) tma_prefetch_map(&tm.q[blockIdx.z]);
    if (FULL && !(BWD && a.o_f32)) tma_prefetch_map(&tm.o[blockIdx.z]);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], FULL ? 2 : 1);
      mbar_init(&s_vfull[s], 1);
      mbar_init(&s_kv[s], 1);
      mbar_init(&s_qs[s], 1);
      mbar_init(&s_pv[s], 1);
      mbar_init(&s_put[s], 256);
      mbar_init(&s_sc[s], 1);
      mbar_init(&s_go[s], 256);
    }
    for (int s = 0; s < 4; ++s) mbar_init(&s_rd[s], 32);
    mbar_init(&s_drain, 1);
    mbar_init(&s_p, 256);
    mbar_init(&s_b, 512);
    mbar_init(&s_pad, 256);
    s_fail = 0;
    s_bad = 0;
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
  if (threadIdx.x >= 64 && threadIdx.x < 64 + kLaT) {
    const int i = (int)threadIdx.x - 64, x = rev ? 32 + i : 127 - i;
    const float g = a.c_out * a.c_kv * (float)la_pow(ld, i);
    s_wt[x] = g;
    if (x > 0) s_wt[kLaWt2 + x - 1] = g;
  } else if (threadIdx.x >= 256 && threadIdx.x < 288) {
    const int x = (int)threadIdx.x - 256 + (rev ? 0 : kLaT);
    s_wt[x] = 0.0f;
    if (x > 0) s_wt[kLaWt2 + x - 1] = 0.0f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_for_launch_before();
  const unsigned tmem = s_tmem;
  const unsigned t_sc = tmem, t_kv = tmem + 256, t_oi = tmem + 448;
  // token of row 0 of the c-th chunk walked, and its number of tokens
  const auto t0 = [&](int c) { return tb + (rev ? nc - 1 - c : c) * kLaT; };
  const int c_tail = rev ? 0 : nc - 1, n_tail = len - (nc - 1) * kLaT;  // the chunk with padding
  const auto rows = [&](int c) { return c == c_tail ? n_tail : kLaT; };

  // whether a chunk's output goes out as one tensor store: bf16, and no row of the
  // tile that must stay as it is (the store clips at L itself)
  const bool tail_staged = n_tail == kLaT || tb + len == p.L, bf16_out = !(BWD && a.o_f32);
  const auto staged = [&](int c) { return bf16_out && (c != c_tail || tail_staged); };

  // the state, and its bf16 copy's halves, belong to warps 10-17
  const int qd = warp & 3, row = 32 * qd + lane, hf = warp < 10 ? (warp - 2) >> 2 : (warp - 10) >> 2;
  const unsigned lane_off = (unsigned)(32 * qd) << 16;
  f32x2 s[16];  // 32 columns of state row `row`, from column cs0
  const int cs0 = col0 + 32 * hf;
  // where this thread's four 16-byte units of row `row` lie in a swizzled block
  unsigned unit[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) unit[j] = sbase + la_unit(0u, row, 4 * hf + j);

  // the update of chunk c: two buffers where no scores are made
  const auto t_up = [&](int c) { return FULL ? t_kv : tmem + 256u * (unsigned)(c & 1); };
  // Weighted v of chunk c, in three (two) pieces: thread = token, half of the columns;
  // vfull, vtail: the token's weight in a full chunk and in the last one.  False where a
  // wait ran out.
  const auto weight = [&](int n) {
    return row < n ? a.c_kv * (float)la_pow(ld, rev ? row + 1 : n - 1 - row) : 0.0f;
  };
  const auto weigh = [&](int c, float vfull, float vtail) {
    const int st = c & 1, n = rows(c);
    bool ok = la_wait(&s_vfull[st], (unsigned)(c >> 1) & 1u, limit);
    if (ok && n < kLaT) ok = la_wait(&s_full[st], (unsigned)(c >> 1) & 1u, limit);
    if (!__all_sync(0xffffffffu, ok)) return false;
    const unsigned vw = FULL || !st ? Sm::kVw : Sm::kVw2;
    const unsigned vb = Sm::kV + st * kLaBlk;
    float f = vfull;
    if (n < kLaT) {
      f = vtail;
      if (row >= n) {  // padding of v and k: whatever it holds becomes zero
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sts128(unit[j] + vb, 0u, 0u, 0u, 0u);
#pragma unroll
          for (int m = 0; m < KD / 64; ++m)
            sts128(unit[j] + Sm::kK + (st * (KD / 64) + m) * kLaBlk, 0u, 0u, 0u, 0u);
        }
      }
    }
    const f32x2 ff = pair2(f, f), minus = pair2(-1.0f, -1.0f);
    uint4 in[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) in[j] = lds128(unit[j] + vb);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned v4[4] = {in[j].x, in[j].y, in[j].z, in[j].w};
      unsigned w1[4], w2[4], w3[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x2 y = mul2(pair2(bf16_lo(v4[g]), bf16_hi(v4[g])), ff);
        float y0, y1, z0, z1;
        unpair2(y, y0, y1);
        w1[g] = pack_bf16(y0, y1);
        const f32x2 z = fma2(pair2(bf16_lo(w1[g]), bf16_hi(w1[g])), minus, y);
        unpair2(z, z0, z1);
        w2[g] = pack_bf16(z0, z1);
        if (three) {
          unpair2(fma2(pair2(bf16_lo(w2[g]), bf16_hi(w2[g])), minus, z), z0, z1);
          w3[g] = pack_bf16(z0, z1);
        }
      }
      sts128(unit[j] + vw, w1[0], w1[1], w1[2], w1[3]);
      sts128(unit[j] + vw + kLaBlk, w2[0], w2[1], w2[2], w2[3]);
      if (three) sts128(unit[j] + vw + 2 * kLaBlk, w3[0], w3[1], w3[2], w3[3]);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    tc_fence_before();
    return true;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---- tensor copies ----------------------------------------------------------
      const CUtensorMap *mq = &tm.q[blockIdx.z], *mk = &tm.k[blockIdx.z], *mv = &tm.v[blockIdx.z];
      const int hq = h / a.q.rep, hk = h / a.k.rep, hv = h / a.v.rep;
      int kin = 0, vin = 0;  // chunks whose k, and whose v, were asked for
      bool ok = true;
      for (int c = 0; c < nc + 2 && !*(volatile int*)&s_fail; ++c) {
        const int st = c & 1;
        const unsigned before = (unsigned)((c >> 1) - 1) & 1u;  // parity of chunk c - 2
        const unsigned sk = sbase + Sm::kK + st * (KD / 64) * kLaBlk,
                       sq = sbase + Sm::kQ + st * (KD / 64) * kLaBlk,
                       sv = sbase + Sm::kV + st * kLaBlk;
        // each buffer as soon as chunk c - 2 has no more use for it: k, q, then v, where
        // that chunk's output is staged
        if (!FULL && c < nc) {  // v is of no use once it has been weighted
          if (c >= 2) ok = la_wait(&s_go[st], before, limit);
          if (!ok) break;
          mbar_expect_tx(&s_vfull[st], kLaBlk);
          tma_load_4d_s(sv, mv, col0, t0(c), hv, b, &s_vfull[st]);
          vin = c + 1;
        }
        if (c < nc) {
          if (c >= 2) ok = la_wait(&s_kv[st], before, limit);
          if (!ok) break;
          mbar_expect_tx(&s_full[st], (KD / 64) * kLaBlk);
#pragma unroll
          for (int j = 0; j < KD / 64; ++j)
            tma_load_4d_s(sk + j * kLaBlk, mk, 64 * j, t0(c), hk, b, &s_full[st]);
          kin = c + 1;
          if (FULL) {
            if (c >= 2) ok = la_wait(&s_qs[st], before, limit);
            if (!ok) {
              mbar_arrive(&s_full[st]);  // in q's place: k alone is waited for below
              break;
            }
            mbar_expect_tx(&s_full[st], (KD / 64) * kLaBlk);
#pragma unroll
            for (int j = 0; j < KD / 64; ++j)
              tma_load_4d_s(sq + j * kLaBlk, mq, 64 * j, t0(c), hq, b, &s_full[st]);
          }
        }
        if (FULL && c >= 2) {
          ok = la_wait(&s_put[st], before, limit);
          if (!ok) break;
          if (staged(c - 2)) {
            tma_store_4d(&tm.o[blockIdx.z], sv, col0, t0(c - 2), h, b);
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          }
        }
        if (FULL && c < nc) {
          mbar_expect_tx(&s_vfull[st], kLaBlk);
          tma_load_4d_s(sv, mv, col0, t0(c), hv, b, &s_vfull[st]);
          vin = c + 1;
        }
        if (c + kLaAhead < nc) {
          const int t = t0(c + kLaAhead);
#pragma unroll
          for (int j = 0; j < KD / 64; ++j) {
            tma_prefetch_4d(mk, 64 * j, t, hk, b);
            if (FULL) tma_prefetch_4d(mq, 64 * j, t, hq, b);
          }
          tma_prefetch_4d(mv, col0, t, hv, b);
        }
      }
      if (!ok) s_fail = 1;  // also where only the last outputs are not stored
      // no copy is in flight when the CTA exits: the last output has been read, and behind it
      // all loads were; the loads of the last two chunks are waited for where there is none
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      if (!FULL || *(volatile int*)&s_fail) {
        const long long last = limit < 2000000000LL ? 2000000000LL : limit;
        for (int i = kin < 2 ? 0 : kin - 2; i < kin; ++i)
          la_wait(&s_full[i & 1], (unsigned)(i >> 1) & 1u, last);
        for (int i = vin < 2 ? 0 : vin - 2; i < vin; ++i)
          la_wait(&s_vfull[i & 1], (unsigned)(i >> 1) & 1u, last);
      }
    }
  } else if (warp == 1) {
    // ---- products -----------------------------------------------------------------
    // descriptors of stage 0; an address enters a descriptor in units of 16 bytes
    const unsigned long long dq0 = umma_desc_sw128(sbase + Sm::kQ),
                             dk0 = umma_desc_sw128(sbase + Sm::kK),
                             dkt0 = umma_desc_mn_sw128(sbase + Sm::kK),
                             dv0 = umma_desc_mn_sw128(sbase + Sm::kV),
                             dw = umma_desc_mn_sw128(sbase + Sm::kVw),
                             ds = umma_desc_mn_sw128(sbase + Sm::kS),
                             dw2 = umma_desc_mn_sw128(sbase + Sm::kVw2) - dw;
    // the whole warp waits; true in every lane or in none
    const auto wait = [&](unsigned long long* bar, unsigned parity) {
      const bool ok = la_wait(bar, parity, limit);
      return __all_sync(0xffffffffu, ok) != 0;
    };
    bool ok = true;
    // Of each chunk the update first (the state's way to the next chunk is the longest),
    // the two outputs, then the scores of the next chunk, which are weighted while its
    // update and carried output are made.
    for (int c = -1; c < nc && !*(volatile int*)&s_fail; ++c) {
      const int st = c & 1;
      const unsigned par = (unsigned)c & 1u, par2 = (unsigned)(c >> 1) & 1u;
      const unsigned stq = st * (KD / 64) * (kLaBlk >> 4);
      if (c >= 0) {
        // weighted v is there, the last update from the same columns has been read
        if (!FULL) ok = wait(&s_full[st], par2) && (c < 2 || wait(&s_put[st], par2 ^ 1u));
        ok = ok && wait(&s_go[st], par2);
        if (!ok) break;
        tc_fence_after();
        if (la_elect()) {
#pragma unroll
          for (int i = 0; i < kLaT / 16; ++i)
            umma_f16_ss(t_up(c), dkt0 + stq + i * 128u, dw + (FULL || !st ? 0u : dw2) + i * 128u,
                        three ? la_idesc(192, true, true) : la_idesc(128, true, true), i != 0);
          umma_commit(&s_kv[st]);
        }
        __syncwarp();
        if (!FULL) continue;
        ok = wait(&s_b, par);  // the state's copy is there, the last outputs have been read
        if (!ok) break;
        tc_fence_after();
        if (la_elect()) {
#pragma unroll
          for (int i = 0; i < KD / 16; ++i)
            umma_f16_ss(t_oi, dq0 + stq + (i >> 2) * (kLaBlk >> 4) + (i & 3) * 2u, ds + i * 128u,
                        la_idesc(64, false, true), i != 0);
          umma_commit(&s_qs[st]);
        }
        __syncwarp();
        ok = wait(&s_p, par);
        if (!ok) break;
        tc_fence_after();
        if (la_elect()) {
#pragma unroll
          for (int i = 0; i < kLaT / 16; ++i)
            umma_f16_ts(t_sc + 128 * st + 64, t_sc + 128 * st + i * 8,
                        dv0 + st * (kLaBlk >> 4) + i * 128u, la_idesc(64, false, true), i != 0);
          umma_commit(&s_pv[st]);
        }
        __syncwarp();
      }
      if (FULL && c + 1 < nc) {
        const int sn = st ^ 1;
        const unsigned stn = sn * (KD / 64) * (kLaBlk >> 4);
        ok = wait(&s_full[sn], (unsigned)((c + 1) >> 1) & 1u);
        // a chunk's padding is cleared before its scores are made
        if (ok && rows(c + 1) < kLaT) ok = wait(&s_pad, 0u);
        if (!ok) break;
        tc_fence_after();
        if (la_elect()) {
#pragma unroll
          for (int i = 0; i < KD / 16; ++i) {
            const unsigned off = stn + (i >> 2) * (kLaBlk >> 4) + (i & 3) * 2u;
            umma_f16_ss(t_sc + 128 * sn, dq0 + off, dk0 + off, la_idesc(128, false, false), i != 0);
          }
          umma_commit(&s_sc[sn]);
        }
        __syncwarp();
      }
    }
    if (!ok) s_fail = 1;
    // every product has completed before the TMEM is given back
    if (la_elect()) umma_commit(&s_drain);
    __syncwarp();
    const long long last = limit < 2000000000LL ? 2000000000LL : limit;
    la_wait(&s_drain, 0u, last);
  } else if (!FULL && warp < 10) {
    // ---- weighted v, one chunk ahead of its product -----------------------------------
    const float vfull = weight(kLaT), vtail = weight(n_tail);
    for (int c = 0; c < nc; ++c) {
      // the place has been read
      bool ok = c < 2 || la_wait(&s_kv[c & 1], (unsigned)((c >> 1) - 1) & 1u, limit);
      ok = __all_sync(0xffffffffu, ok) && weigh(c, vfull, vtail);
      if (!ok) {
        s_fail = 1;
        break;
      }
      mbar_arrive(&s_go[c & 1]);
    }
  } else if (warp < 10) {
    // ---- weighted scores and outputs: thread = token, half of the columns -----------
    const int i = row;
    const long long obase = (long long)b * a.ob + (long long)h * a.oh + col0;
    const int nd = a.dv - col0 < kLaN ? a.dv - col0 : kLaN;
    const bool f32 = BWD && a.o_f32;
    // this row's factor of the carried output, in a full chunk and in the last one
    const float e_full = a.c_out * (float)la_pow(ld, rev ? kLaT - 1 - i : i + 1);
    const float e_tail =
        i < n_tail ? a.c_out * (float)la_pow(ld, rev ? n_tail - 1 - i : i + 1) : 0.0f;
    const int x0 = rev ? 32 - i : 127 - i;
    const float* wt0 = s_wt + (x0 & 1 ? kLaWt2 + x0 - 1 : x0);
    unsigned big = 0u;  // the largest of this token's weighted scores, two columns at a time
    if (nc > 0) mbar_arrive(&s_b);  // chunk 0 has no outputs before it
    for (int c = 0; c < nc; ++c) {
      const int st = c & 1;
      const unsigned par = (unsigned)c & 1u, par2 = (unsigned)(c >> 1) & 1u;
      const int n = rows(c);
      bool ok = la_wait(&s_sc[st], par2, limit);
      if (!__all_sync(0xffffffffu, ok)) {
        s_fail = 1;
        break;
      }
      tc_fence_after();
      const unsigned t_s = t_sc + lane_off + 128 * st;
      // two blocks of 32 columns; those beyond the diagonal block J = qd are zero
      unsigned w[32], most = big;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        const int J = 2 * hf + jj;
        if (rev ? J >= qd : J <= qd) {  // uniform in the warp
          unsigned r[32];
          tmem_ld16_async(t_s + 32 * J, r);
          tmem_ld16_async(t_s + 32 * J + 16, r + 16);
          f32x2 f[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            f[e] = *reinterpret_cast<const f32x2*>(wt0 + 32 * J + 2 * e);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float y0, y1;
            unpair2(mul2(pair2u(r[2 * e], r[2 * e + 1]), f[e]), y0, y1);
            w[16 * jj + e] = pack_bf16(y0, y1);
            most = larger_bf16x2(most, w[16 * jj + e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[16 * jj + e] = 0u;
        }
      }
      if (i < n) big = most;
      // the weighted scores go to columns 0-63, where the warp of the lower half reads
      tc_fence_before();
      if (hf == 0) {
        mbar_arrive(&s_rd[qd]);
      } else {
        ok = la_wait(&s_rd[qd], par, limit);
        if (!__all_sync(0xffffffffu, ok)) {
          s_fail = 1;
          break;
        }
        tc_fence_after();
      }
      tmem_st16(t_s + 32 * hf, w);
      tmem_st16(t_s + 32 * hf + 16, w + 16);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&s_p);

      ok = la_wait(&s_pv[st], par2, limit);
      if (!__all_sync(0xffffffffu, ok)) {
        s_fail = 1;
        break;
      }
      tc_fence_after();
      unsigned y[32];
      tmem_ld16_async(t_oi + lane_off + 32 * hf, y);
      tmem_ld16_async(t_s + 64 + 32 * hf, w);
      tmem_ld16_async(t_oi + lane_off + 32 * hf + 16, y + 16);
      tmem_ld16_async(t_s + 64 + 32 * hf + 16, w + 16);
      const float e = c == c_tail ? e_tail : e_full;
      const f32x2 ee = pair2(e, e);
      tmem_wait_ld();
      tc_fence_before();
      if (c + 1 < nc) mbar_arrive(&s_b);  // chunk c + 1 may write the outputs
      f32x2 x[16];
#pragma unroll
      for (int d = 0; d < 16; ++d)
        x[d] = fma2(ee, pair2u(y[2 * d], y[2 * d + 1]), pair2u(w[2 * d], w[2 * d + 1]));
      if (staged(c)) {
        const unsigned ob = Sm::kV + st * kLaBlk;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          unsigned u[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float x0, x1;
            unpair2(x[4 * d + g], x0, x1);
            u[g] = pack_bf16(x0, x1);
          }
          sts128(unit[d] + ob, u[0], u[1], u[2], u[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      } else if (i < n) {
        const long long at = obase + (long long)(t0(c) + i) * a.ot + 32 * hf;
#pragma unroll
        for (int d = 0; d < 32; d += 4)
          if (32 * hf + d < nd) {
            float4 y4;
            unpair2(x[d / 2], y4.x, y4.y);
            unpair2(x[d / 2 + 1], y4.z, y4.w);
            if (f32)
              *reinterpret_cast<float4*>(static_cast<float*>(a.o) + at + d) = y4;
            else
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + at + d) =
                  make_uint2(pack_bf16(y4.x, y4.y), pack_bf16(y4.z, y4.w));
          }
      }
      mbar_arrive(&s_put[st]);
    }
    if ((big & 0x7F80u) == 0x7F80u || (big & 0x7F800000u) == 0x7F800000u) s_bad = 1;
    if (p.zero_tail && !*(volatile int*)&s_fail) {
      const long long end = span == p.nspan - 1 ? p.L : tb + p.span;
      for (long long t = (long long)tb + len + i; t < end; t += kLaT)
        for (int d = 8 * hf; d < nd; d += 16) {
          const long long at = obase + t * a.ot + d;
          const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
          if (f32) {
            *reinterpret_cast<uint4*>(static_cast<float*>(a.o) + at) = zero;
            *reinterpret_cast<uint4*>(static_cast<float*>(a.o) + at + 4) = zero;
          } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + at) = zero;
          }
        }
    }
  } else {
    // ---- the state and weighted v: thread = state row = token, half of the columns -----
    const int r = row;
#pragma unroll
    for (int d = 0; d < 16; ++d) s[d] = 0;
    if (s_in && r < a.dk) {
      const float* sp = s_in + sb + r * sr + cs0 * sc;
      if (sc == 1) {  // pairs as they lie, waited for where the state is first used
#pragma unroll
        for (int d = 0; d < 32; d += 4)
          if (cs0 + d < a.dv) {
            const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(sp + d);
            s[d / 2] = two.x;
            s[d / 2 + 1] = two.y;
          }
      } else {  // transposed: the lanes' rows are neighbours
#pragma unroll
        for (int d = 0; d < 32; d += 2)
          if (cs0 + d < a.dv) s[d / 2] = pair2(sp[d * sc], sp[(d + 1) * sc]);
      }
    }
    float ghi, glo;  // gamma^128
    la_two(ld, kLaT, ghi, glo);
    const float vfull = FULL ? weight(kLaT) : 0.0f, vtail = FULL ? weight(n_tail) : 0.0f;
    bool ok = true;
    for (int c = 0; c <= nc; ++c) {
      const int st = c & 1;
      if (c > 0) {
        // s <- gamma^m s + U of the chunk before, which had m tokens
        ok = la_wait(&s_kv[st ^ 1], (unsigned)((c - 1) >> 1) & 1u, limit);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float h1 = ghi, h2 = glo;
        const int m = rows(c - 1);
        if (m < kLaT) la_two(ld, m, h1, h2);
        const f32x2 hh1 = pair2(h1, h1), hh2 = pair2(h2, h2);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          unsigned u1[16], u2[16], u3[16];
          const unsigned t_u = t_up(c - 1) + lane_off + 32 * hf + 16 * part;
          tmem_ld16_async(t_u, u1);
          tmem_ld16_async(t_u + 64, u2);
          if (three) tmem_ld16_async(t_u + 128, u3);
          tmem_wait_ld();
#pragma unroll
          for (int d = 0; d < 8; ++d) {
            const f32x2 old = s[8 * part + d];
            f32x2 low = pair2u(u2[2 * d], u2[2 * d + 1]);
            if (three) low = add2(low, pair2u(u3[2 * d], u3[2 * d + 1]));
            low = fma2(hh2, old, low);
            s[8 * part + d] = fma2(hh1, old, add2(pair2u(u1[2 * d], u1[2 * d + 1]), low));
          }
        }
      }
      if (!FULL && c > 0) {
        tc_fence_before();
        mbar_arrive(&s_put[st ^ 1]);
      }
      if (c == nc) break;
      if (!FULL) continue;
      if (!weigh(c, vfull, vtail)) {
        ok = false;
        break;
      }
      mbar_arrive(&s_go[st]);
      if (rows(c) < kLaT) mbar_arrive(&s_pad);
      if (c > 0) {  // the last copy of the state has been read
        ok = la_wait(&s_qs[st ^ 1], (unsigned)((c - 1) >> 1) & 1u, limit);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
      }
      if (KD == 128 || r < KD) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          unsigned u[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float x0, x1;
            unpair2(s[4 * j + g], x0, x1);
            u[g] = pack_bf16(x0, x1);
          }
          sts128(unit[j] + Sm::kS, u[0], u[1], u[2], u[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&s_b);
    }
    if (!ok) {
      s_fail = 1;
    } else if (r < a.dk) {
      bool fine = true;
#pragma unroll
      for (int d = 0; d < 16; ++d) {
        float x0, x1;
        unpair2(s[d], x0, x1);
        fine = fine && isfinite(x0) && isfinite(x1);  // columns past dv are sums of zeros
      }
      if (!fine) s_bad = 1;
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
  if (s_fail) return;
  if (s_bad) {  // the outputs of a walk of the states only are replaced by the full one's
    if (threadIdx.x == 0)  // the outputs stored so far are there before others replace them
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncthreads();
    if (threadIdx.x < kLaAgainThreads)
      la_walk<kLaN, kLaAgainThreads>(
          p, a, b, h, col0, tb, len, s_in ? s_in + sb : nullptr, sr, sc,
          s_out ? s_out + sb : nullptr, *reinterpret_cast<LaWalkSmem<kLaN>*>(dsmem));
  } else if (warp >= 10 && s_out) {
    // through shared memory (nothing uses q's place any more), so that 16 lanes store one
    // row: stored straight from the rows' threads, 128 x 64 states took 3100 cycles
#pragma unroll
    for (int d = 0; d < 32; d += 4) {
      float4 x;
      unpair2(s[d / 2], x.x, x.y);
      unpair2(s[d / 2 + 1], x.z, x.w);
      if (KD == 128 || row < KD)
        sts128(sbase + Sm::kQ + row * 256 + (((8 * hf + d / 4) ^ (row & 15)) << 4),
               __float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z),
               __float_as_uint(x.w));
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
    for (int i = 0; i < KD / 16; ++i) {
      const int at = (int)threadIdx.x - 320 + 256 * i, to = at >> 4, u = at & 15;
      if (to < a.dk && col0 + 4 * u < a.dv)
        *reinterpret_cast<uint4*>(s_out + sb + (long long)to * a.dv + col0 + 4 * u) =
            lds128(sbase + Sm::kQ + to * 256 + ((u ^ (to & 15)) << 4));
    }
  }
}

// The states that the spans' own tokens leave (s_span, [B, H, spans, dk, dv]) become the
// states before the spans; the state behind the last one goes to s_out.  A thread an
// element, eight spans' loads on their way at a time.  With eight elements a thread, one
// load after the other and launches that do not overlap, a scan of 16 spans of 8 heads of
// 64 took 39 us, with this 21.
constexpr int kLaJoinThreads = 256;
constexpr int kLaJoinAhead = 8;  // spans whose states are on their way at a time

__global__ void __launch_bounds__(kLaJoinThreads)
    pararnn_linattn_join_kernel(const __grid_constant__ LaParams p) {
  const LaPass& a = p.pass[blockIdx.z];
  const int bh = blockIdx.x, b = bh / p.H;
  const float ld = p.log_decay[bh % p.H];
  const int n = a.dk * a.dv, e = (int)(threadIdx.x + blockIdx.y * kLaJoinThreads);
  float ghi, glo;  // of a whole span
  la_two(ld, p.span, ghi, glo);
  wait_for_launch_before();
  if (e >= n) return;
  const int r = e / a.dv, c = e % a.dv;
  float x = a.s_in ? a.s_in[(long long)bh * n + r * a.s_r + c * a.s_c] : 0.0f;
  float* sp = a.s_span + (long long)bh * p.nspan * n + e;
  for (int k0 = 0; k0 < p.nspan; k0 += kLaJoinAhead) {
    float own[kLaJoinAhead];
#pragma unroll
    for (int i = 0; i < kLaJoinAhead; ++i)
      if (k0 + i < p.nspan)
        own[i] = sp[(long long)(a.rev ? p.nspan - 1 - k0 - i : k0 + i) * n];
#pragma unroll
    for (int i = 0; i < kLaJoinAhead; ++i) {
      if (k0 + i >= p.nspan) break;
      const int g = a.rev ? p.nspan - 1 - k0 - i : k0 + i;
      const long long m = la_span_tokens(p, b, g);
      float h1 = ghi, h2 = glo;
      if (m != p.span) la_two(ld, m, h1, h2);
      sp[(long long)g * n] = x;
      x = m == 0 ? x : fmaf(h1, x, fmaf(h2, x, own[i]));
    }
  }
  if (a.s_out) a.s_out[(long long)bh * n + e] = x;
}

}  // namespace pararnn
