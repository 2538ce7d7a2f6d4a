// linattn.cu -- C ABI of the linear-attention operators (declared in
// include/pararnn.h): argument validation, workspace layout and launches.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include <cudaTypedefs.h>

#include "pararnn.h"
#include "pararnn_linattn.cuh"
#include "pararnn_linattn_chunk.cuh"

namespace pararnn {
namespace {

bool la_aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

size_t la_round(size_t n) { return (n + 511) / 512 * 512; }  // more than kLaNoWs

bool la_sizes_ok(const pararnn_linattn_t* d) {
  if (!d || d->B < 0 || d->L < 0 || d->H <= 0 || d->Hq <= 0 || d->Hk <= 0 || d->Hv <= 0)
    return false;
  if (d->H % d->Hq || d->H % d->Hk || d->H % d->Hv) return false;
  if (d->Dk <= 0 || d->Dv <= 0 || d->Dk % 8 || d->Dv % 8 || d->Dk > kLaMaxDim || d->Dv > kLaMaxDim)
    return false;
  if (d->L >= (1LL << 31) - 256 || d->B > (1LL << 31) - 1 || d->H > (1 << 20)) return false;
  if (d->B * d->H >= (1LL << 31) - 1) return false;
  return std::isfinite(d->scale);
}

// Strides of a stream: tensor copies need whole 16-byte units (8 bf16).
bool la_strides_ok(const int64_t* s) {
  for (int i = 0; i < 3; ++i)
    if (s[i] <= 0 || s[i] % 8 || s[i] >= (1LL << 38)) return false;
  return true;
}

LaIn la_in(const void* p, const int64_t* s, int H, int Hx) {
  return LaIn{p, s[0], s[1], s[2], H / Hx};
}

pararnn_status_t la_launch_recurrent(const LaParams& lp, cudaStream_t st) {
  int dv = 0;
  for (int i = 0; i < lp.npass; ++i) dv = lp.pass[i].dv > dv ? lp.pass[i].dv : dv;
  const dim3 grid((unsigned)((long long)lp.B * lp.H), (unsigned)((dv + 31) / 32),
                  (unsigned)lp.npass);
  pararnn_linattn_recurrent_kernel<<<grid, kLaRecThreads, 0, st>>>(lp);
  return cudaGetLastError() == cudaSuccess ? PARARNN_OK : PARARNN_ERR_CUDA;
}

std::once_flag g_la_once;
PFN_cuTensorMapEncodeTiled_v12000 g_la_encode = nullptr;

PFN_cuTensorMapEncodeTiled_v12000 la_encoder() {
  std::call_once(g_la_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_la_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    else
      cudaGetLastError();
  });
  return g_la_encode;
}

// A stream [B, L, Hx, D] as a 4-D tensor {D, L, Hx, B}: boxes of 64 columns (one
// 128-byte swizzle row) x 128 tokens of one head; what lies outside reads as zero.
bool la_map(CUtensorMap* m, const void* base, long long st, long long sh, long long sb, int D,
            int Hx, const LaParams& lp) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = la_encoder();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)lp.L, (cuuint64_t)Hx, (cuuint64_t)lp.B};
  const cuuint64_t strides[3] = {(cuuint64_t)st * 2, (cuuint64_t)sh * 2, (cuuint64_t)sb * 2};
  const cuuint32_t box[4] = {64, kLaT, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool la_map(CUtensorMap* m, const LaIn& in, int D, const LaParams& lp) {
  return la_map(m, in.p, in.st, in.sh, in.sb, D, lp.H / in.rep, lp);
}

template <int KD, bool FULL, bool BWD>
pararnn_status_t la_launch_chunk(const LaParams& lp, const LaMaps& tm, cudaStream_t st) {
  // the kernel's shared memory has been raised on these devices (by index)
  static std::atomic<unsigned long long> raised{0};
  const void* fn = (const void*)pararnn_linattn_chunk_kernel<KD, FULL, BWD>;
  const size_t smem = LaSmem<KD>::bytes(FULL);
  int dv = 0;
  for (int i = 0; i < lp.npass; ++i) dv = lp.pass[i].dv > dv ? lp.pass[i].dv : dv;
  const dim3 grid((unsigned)((long long)lp.B * lp.H * lp.nspan),
                  (unsigned)((dv + kLaN - 1) / kLaN), (unsigned)lp.npass);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PARARNN_ERR_CUDA;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  // a second try where the first launch is refused: a device that was reset since has
  // forgotten the setting
  for (bool known = (raised.load(std::memory_order_relaxed) & bit) != 0;; known = false) {
    if (!known) {
      const cudaError_t e =
          cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) {
        cudaGetLastError();
        return e == cudaErrorNoKernelImageForDevice || e == cudaErrorInvalidDeviceFunction
                   ? PARARNN_ERR_UNSUPPORTED
                   : PARARNN_ERR_CUDA;
      }
      raised.fetch_or(bit, std::memory_order_relaxed);
    }
    if (FULL && lp.nspan > 1)  // behind the join
      launch_behind(pararnn_linattn_chunk_kernel<KD, FULL, BWD>, grid, dim3(kLaThreads), smem, st,
                    lp, tm);
    else
      pararnn_linattn_chunk_kernel<KD, FULL, BWD><<<grid, kLaThreads, smem, st>>>(lp, tm);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return PARARNN_OK;
    if (!known) return PARARNN_ERR_CUDA;
  }
}

// The launches of one call.
template <int KD>
pararnn_status_t la_walks(const LaParams& lp, const LaMaps& tm, cudaStream_t st) {
  if (lp.nspan > 1) {
    const pararnn_status_t rc = lp.npass > 1 ? la_launch_chunk<KD, false, true>(lp, tm, st)
                                             : la_launch_chunk<KD, false, false>(lp, tm, st);
    if (rc != PARARNN_OK) return rc;
    int n = 0;
    for (int i = 0; i < lp.npass; ++i) n = lp.pass[i].dk * lp.pass[i].dv;  // the same in all
    const dim3 grid((unsigned)((long long)lp.B * lp.H),
                    (unsigned)((n + kLaJoinThreads - 1) / kLaJoinThreads), (unsigned)lp.npass);
    if (launch_behind(pararnn_linattn_join_kernel, grid, dim3(kLaJoinThreads), 0, st, lp) !=
        cudaSuccess) {
      cudaGetLastError();
      return PARARNN_ERR_CUDA;
    }
  }
  return lp.npass > 1 ? la_launch_chunk<KD, true, true>(lp, tm, st)
                      : la_launch_chunk<KD, true, false>(lp, tm, st);
}

// The form of a call and, for the chunked form, the spans that time is cut into.
// The recurrent form's time grows with every token, the chunked one's with every 128.
// Scan, one launch in a graph, recurrent / chunked: one sequence of 8 heads of 128 at 8
// tokens 8.7 / 8.4 us, at 16 14.2 / 8.6; 8 x 16 heads of 128 at 8 tokens 14.2 / 16.9, at
// 16 23.9 / 16.8; 32 x 16 heads of 64 at 8 tokens 17.0 / 29.2, at 16 27.9 / 29.2.
constexpr long long kLaRecurrentMax = 8;
constexpr long long kLaSms = 148;  // one CTA of the chunked form each

struct LaPlan {
  bool recurrent;
  int nspan;
  long long span;  // tokens
};

LaPlan la_plan(const pararnn_linattn_t* d, bool backward, const pararnn_options_t* opts) {
  const int form = opts ? opts->regime : 0;
  LaPlan pl = {form == 1 || (form == 0 && d->L <= kLaRecurrentMax), 1, d->L};
  if (pl.recurrent) return pl;
  const long long tk = (d->Dk + kLaN - 1) / kLaN, tv = (d->Dv + kLaN - 1) / kLaN;
  const long long items = d->B * d->H * (backward ? 2 * tk + tv : tv);
  const long long chunks = (d->L + kLaT - 1) / kLaT;
  if (items >= 4 * kLaSms) return pl;
  // In units of one chunk's walk (2 us): a CTA takes about two to start and end.  With more
  // than one span the states are walked first, 0.45 a chunk, and the join and two more
  // launches take 4 to 7.  Measured in us, one span and the best number of them: 2048 tokens of
  // 8 heads of 64 38, 18 (16 spans); 4096 of 16 heads of 128 68, 46 (4); 65536 of 12
  // heads of 64 1014, 149 (12); 4 x 4096 of 8 heads of 128 70, 77 (2: not taken).
  const double join = d->Dk * d->Dv <= 64 * 64 ? 4.0 : 7.0;
  double best = 0.0;
  for (long long want = 1; want <= chunks && (want - 1) * items <= 2 * kLaSms; ++want) {
    const long long len = (chunks + want - 1) / want, n = (chunks + len - 1) / len;
    const long long waves = (items * n + kLaSms - 1) / kLaSms;
    const double cost = n > 1 ? waves * (1.45 * len + 4.0) + join : waves * (len + 2.0);
    if (want == 1 || cost < best) {
      best = cost;
      pl.nspan = (int)n;
      pl.span = n > 1 ? len * kLaT : d->L;
    }
  }
  return pl;
}

pararnn_status_t la_launch(LaParams& lp, const LaPlan& pl, float* span_ws,
                           const pararnn_options_t* opts, int32_t* status_dev, cudaStream_t st) {
  lp.nspan = pl.nspan;
  lp.span = pl.span;
  if (pl.recurrent) return la_launch_recurrent(lp, st);
  if (pl.nspan > 1)
    for (int i = 0; i < lp.npass; ++i) {
      lp.pass[i].s_span = span_ws;
      span_ws += (size_t)lp.B * lp.H * pl.nspan * lp.pass[i].dk * lp.pass[i].dv;
    }
  lp.status_dev = status_dev;
  lp.timeout_ns = opts && opts->wait_timeout_ns > 0 ? opts->wait_timeout_ns : 1000000000LL;
  LaMaps tm = {};
  int dk = 0;
  for (int i = 0; i < lp.npass; ++i) {
    const LaPass& a = lp.pass[i];
    if (!la_map(&tm.q[i], a.q, a.dk, lp) || !la_map(&tm.k[i], a.k, a.dk, lp) ||
        !la_map(&tm.v[i], a.v, a.dv, lp) ||
        (!a.o_f32 && !la_map(&tm.o[i], a.o, a.ot, a.oh, a.ob, a.dv, lp.H, lp)))
      return PARARNN_ERR_INVALID_ARGUMENT;
    dk = a.dk > dk ? a.dk : dk;
  }
  return dk <= 64 ? la_walks<64>(lp, tm, st) : la_walks<128>(lp, tm, st);
}

// Tiles of 4096 elements, 4 rows a thread: 128 rows x 32 columns, or 64 x 64 (with 32
// columns half of the threads would have no rows: 256 x 32 states of 64 x 64 76 us, so 45).
template <typename T>
void la_launch_step(const LaParams& lp, unsigned grid, cudaStream_t st) {
  const int dk = lp.pass[0].dk;
  if (dk == 128)
    pararnn_linattn_step_kernel<T, 32, 128, false><<<grid, kLaStepThreads, 0, st>>>(lp);
  else if (dk > 64)
    pararnn_linattn_step_kernel<T, 32, 128, true><<<grid, kLaStepThreads, 0, st>>>(lp);
  else if (dk == 64)
    pararnn_linattn_step_kernel<T, 64, 64, false><<<grid, kLaStepThreads, 0, st>>>(lp);
  else
    pararnn_linattn_step_kernel<T, 64, 64, true><<<grid, kLaStepThreads, 0, st>>>(lp);
}

// Workspace: fp32 per-head gradients of the streams whose heads are shared, and
// the spans' states of every pass.
constexpr size_t kLaNoWs = 256;  // what the size says where a call needs none

struct LaWs {
  size_t dq, dk, dv, span, total;
};
LaWs la_ws(const pararnn_linattn_t* d, bool backward, const LaPlan& pl) {
  LaWs w = {};
  size_t at = 0;
  const size_t rows = (size_t)d->B * (size_t)d->L * (size_t)d->H;
  if (backward) {
    w.dq = at;
    if (d->Hq != d->H) at += la_round(rows * d->Dk * 4);
    w.dk = at;
    if (d->Hk != d->H) at += la_round(rows * d->Dk * 4);
    w.dv = at;
    if (d->Hv != d->H) at += la_round(rows * d->Dv * 4);
  }
  w.span = at;
  if (pl.nspan > 1)
    at += la_round((size_t)(backward ? 3 : 1) * d->B * d->H * pl.nspan * d->Dk * d->Dv * 4);
  w.total = at ? at : kLaNoWs;
  return w;
}

pararnn_status_t la_group(const float* x, void* y, const pararnn_linattn_t* d, int Hx, int D,
                          cudaStream_t st) {
  const long long rows = d->B * d->L;
  const long long n = rows * Hx * (D / 4);
  long long blocks = (n + 255) / 256;
  if (blocks > 148 * 16) blocks = 148 * 16;
  pararnn_linattn_group_kernel<<<(unsigned)blocks, 256, 0, st>>>(
      x, static_cast<__nv_bfloat16*>(y), rows, d->H, Hx, D);
  return cudaGetLastError() == cudaSuccess ? PARARNN_OK : PARARNN_ERR_CUDA;
}

// L = 0: the state passes through unchanged.
pararnn_status_t la_copy_state(const float* s0, float* s, size_t n, cudaStream_t st) {
  if (!s || s == s0 || n == 0) return PARARNN_OK;
  const cudaError_t e = s0 ? cudaMemcpyAsync(s, s0, n * 4, cudaMemcpyDeviceToDevice, st)
                           : cudaMemsetAsync(s, 0, n * 4, st);
  return e == cudaSuccess ? PARARNN_OK : PARARNN_ERR_CUDA;
}

}  // namespace
}  // namespace pararnn

using namespace pararnn;

extern "C" size_t pararnn_linattn_workspace_size(const pararnn_linattn_t* d, int32_t backward) {
  if (!la_sizes_ok(d)) return 0;
  return la_ws(d, backward != 0, la_plan(d, backward != 0, nullptr)).total;
}

extern "C" pararnn_status_t pararnn_scan_linattn(const pararnn_linattn_t* d, const void* q,
                                                 const void* k, const void* v,
                                                 const float* log_decay, const float* s0,
                                                 const int32_t* lengths, void* o, float* s,
                                                 void* ws, size_t ws_bytes, int32_t* status_dev,
                                                 const pararnn_options_t* opts, void* stream) {
  if (!la_sizes_ok(d)) return PARARNN_ERR_INVALID_ARGUMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->B > 0 && d->L > 0) {
    if (!q || !k || !v || !o || !log_decay) return PARARNN_ERR_INVALID_ARGUMENT;
    if (!la_strides_ok(d->q_stride) || !la_strides_ok(d->k_stride) || !la_strides_ok(d->v_stride))
      return PARARNN_ERR_INVALID_ARGUMENT;
    if (!la_aligned(q, 16) || !la_aligned(k, 16) || !la_aligned(v, 16) || !la_aligned(o, 16) ||
        !la_aligned(log_decay, 4) || !la_aligned(lengths, 4))
      return PARARNN_ERR_INVALID_ARGUMENT;
  }
  if (!la_aligned(s0, 16) || !la_aligned(s, 16) || !la_aligned(status_dev, 4))
    return PARARNN_ERR_INVALID_ARGUMENT;
  if (opts && (opts->regime < 0 || opts->regime > 2)) return PARARNN_ERR_INVALID_ARGUMENT;
  const LaPlan pl = la_plan(d, false, opts);
  const LaWs w = la_ws(d, false, pl);
  if (w.total > kLaNoWs && (!ws || ws_bytes < w.total || !la_aligned(ws, 256)))
    return PARARNN_ERR_WORKSPACE;
  if (status_dev && cudaMemsetAsync(status_dev, 0, sizeof(int32_t), st) != cudaSuccess)
    return PARARNN_ERR_CUDA;
  if (d->B == 0) return PARARNN_OK;
  if (d->L == 0)
    return la_copy_state(s0, s, (size_t)d->B * d->H * d->Dk * d->Dv, st);

  LaParams lp = {};
  lp.npass = 1;
  lp.log_decay = log_decay;
  lp.lengths = lengths;
  lp.B = (int)d->B;
  lp.H = d->H;
  lp.L = d->L;
  LaPass& a = lp.pass[0];
  a.q = la_in(q, d->q_stride, d->H, d->Hq);
  a.k = la_in(k, d->k_stride, d->H, d->Hk);
  a.v = la_in(v, d->v_stride, d->H, d->Hv);
  a.o = o;
  a.oh = d->Dv;
  a.ot = (long long)d->H * d->Dv;
  a.ob = a.ot * d->L;
  a.s_in = s0;
  a.s_out = s;
  a.s_r = d->Dv;
  a.s_c = 1;
  a.dk = d->Dk;
  a.dv = d->Dv;
  a.c_out = d->scale;
  a.c_kv = 1.0f;
  return la_launch(lp, pl, static_cast<float*>(ws), opts, status_dev, st);
}

extern "C" pararnn_status_t pararnn_scan_linattn_backward(
    const pararnn_linattn_t* d, const void* q, const void* k, const void* v,
    const float* log_decay, const float* s0, const void* dout, const float* ds,
    const int32_t* lengths, void* dq, void* dk, void* dv, float* ds0, void* ws, size_t ws_bytes,
    int32_t* status_dev, const pararnn_options_t* opts, void* stream) {
  if (!la_sizes_ok(d)) return PARARNN_ERR_INVALID_ARGUMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->B > 0 && d->L > 0) {
    if (!q || !k || !v || !dout || !dq || !dk || !dv || !log_decay)
      return PARARNN_ERR_INVALID_ARGUMENT;
    if (!la_strides_ok(d->q_stride) || !la_strides_ok(d->k_stride) ||
        !la_strides_ok(d->v_stride) || !la_strides_ok(d->do_stride))
      return PARARNN_ERR_INVALID_ARGUMENT;
    const void* ps[] = {q, k, v, dout, dq, dk, dv};
    for (const void* x : ps)
      if (!la_aligned(x, 16)) return PARARNN_ERR_INVALID_ARGUMENT;
    if (!la_aligned(log_decay, 4) || !la_aligned(lengths, 4)) return PARARNN_ERR_INVALID_ARGUMENT;
  }
  if (!la_aligned(s0, 16) || !la_aligned(ds, 16) || !la_aligned(ds0, 16) || (ds && ds == ds0) ||
      !la_aligned(status_dev, 4))
    return PARARNN_ERR_INVALID_ARGUMENT;
  if (opts && (opts->regime < 0 || opts->regime > 2)) return PARARNN_ERR_INVALID_ARGUMENT;
  const LaPlan pl = la_plan(d, true, opts);
  const LaWs w = la_ws(d, true, pl);
  if (w.total > kLaNoWs && (!ws || ws_bytes < w.total || !la_aligned(ws, 256)))
    return PARARNN_ERR_WORKSPACE;
  if (status_dev && cudaMemsetAsync(status_dev, 0, sizeof(int32_t), st) != cudaSuccess)
    return PARARNN_ERR_CUDA;
  if (d->B == 0) return PARARNN_OK;
  if (d->L == 0)
    return la_copy_state(ds, ds0, (size_t)d->B * d->H * d->Dk * d->Dv, st);

  unsigned char* wb = static_cast<unsigned char*>(ws);
  LaParams lp = {};
  lp.npass = 3;
  lp.log_decay = log_decay;
  lp.lengths = lengths;
  lp.B = (int)d->B;
  lp.H = d->H;
  lp.L = d->L;
  lp.zero_tail = 1;
  const LaIn iq = la_in(q, d->q_stride, d->H, d->Hq), ik = la_in(k, d->k_stride, d->H, d->Hk),
             iv = la_in(v, d->v_stride, d->H, d->Hv),
             io = la_in(dout, d->do_stride, d->H, d->H);
  const struct {
    LaIn q, k, v;
    void* out;
    size_t off;
    int Hx, dk, dv, rev;
    const float* s_in;
  } def[3] = {
      {io, iv, ik, dq, w.dq, d->Hq, d->Dv, d->Dk, 0, s0},   // dq
      {iv, io, iq, dk, w.dk, d->Hk, d->Dv, d->Dk, 1, ds},   // dk
      {ik, iq, io, dv, w.dv, d->Hv, d->Dk, d->Dv, 1, ds},   // dv
  };
  for (int i = 0; i < 3; ++i) {
    LaPass& a = lp.pass[i];
    a.q = def[i].q;
    a.k = def[i].k;
    a.v = def[i].v;
    a.dk = def[i].dk;
    a.dv = def[i].dv;
    a.rev = def[i].rev;
    a.o_f32 = def[i].Hx != d->H;
    a.o = a.o_f32 ? (void*)(wb + def[i].off) : def[i].out;
    a.oh = a.dv;
    a.ot = (long long)d->H * a.dv;
    a.ob = a.ot * d->L;
    a.s_in = def[i].s_in;
    a.s_out = i == 2 ? ds0 : nullptr;
    // states are stored [Dk, Dv]; the dq and dk passes carry the transpose
    a.s_r = i == 2 ? d->Dv : 1;
    a.s_c = i == 2 ? 1 : d->Dv;
    a.c_out = i == 0 ? d->scale : 1.0f;
    a.c_kv = i == 0 ? 1.0f : d->scale;
  }
  pararnn_status_t rc =
      la_launch(lp, pl, reinterpret_cast<float*>(wb + w.span), opts, status_dev, st);
  for (int i = 0; i < 3 && rc == PARARNN_OK; ++i)
    if (lp.pass[i].o_f32)
      rc = la_group(static_cast<const float*>(lp.pass[i].o), def[i].out, d, def[i].Hx,
                    lp.pass[i].dv, st);
  return rc;
}

extern "C" pararnn_status_t pararnn_step_linattn(const pararnn_linattn_t* d, const void* q,
                                                 const void* k, const void* v,
                                                 pararnn_dtype_t dtype, const float* log_decay,
                                                 const float* s_prev, void* o, float* s_next,
                                                 void* stream) {
  if (!la_sizes_ok(d) || d->L != 1) return PARARNN_ERR_INVALID_ARGUMENT;
  if (dtype != PARARNN_F32 && dtype != PARARNN_BF16) return PARARNN_ERR_INVALID_ARGUMENT;
  if (d->B == 0) return PARARNN_OK;
  if (!q || !k || !v || !o || !log_decay || !s_next) return PARARNN_ERR_INVALID_ARGUMENT;
  for (const int64_t* x : {d->q_stride, d->k_stride, d->v_stride})
    if (x[0] < 0 || x[2] < 0) return PARARNN_ERR_INVALID_ARGUMENT;
  const size_t es = dtype == PARARNN_F32 ? 4 : 2;
  if (!la_aligned(q, es) || !la_aligned(k, es) || !la_aligned(v, es) || !la_aligned(o, es) ||
      !la_aligned(log_decay, 4) || !la_aligned(s_prev, 16) || !la_aligned(s_next, 16))
    return PARARNN_ERR_INVALID_ARGUMENT;
  LaParams lp = {};
  lp.npass = 1;
  lp.log_decay = log_decay;
  lp.B = (int)d->B;
  lp.H = d->H;
  lp.L = 1;
  lp.nspan = 1;
  lp.span = 1;
  LaPass& a = lp.pass[0];
  a.q = la_in(q, d->q_stride, d->H, d->Hq);
  a.k = la_in(k, d->k_stride, d->H, d->Hk);
  a.v = la_in(v, d->v_stride, d->H, d->Hv);
  a.o = o;
  a.oh = d->Dv;
  a.ot = 0;
  a.ob = (long long)d->H * d->Dv;
  a.s_in = s_prev;
  a.s_out = s_next;
  a.s_r = d->Dv;
  a.s_c = 1;
  a.dk = d->Dk;
  a.dv = d->Dv;
  a.o_f32 = dtype == PARARNN_F32;
  a.c_out = d->scale;
  a.c_kv = 1.0f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long cols = d->Dk <= 64 ? 64 : 32, grid = d->B * d->H * ((d->Dv + cols - 1) / cols);
  if (grid >= (1LL << 31)) return PARARNN_ERR_INVALID_ARGUMENT;
  if (dtype == PARARNN_BF16)
    la_launch_step<__nv_bfloat16>(lp, (unsigned)grid, st);
  else
    la_launch_step<float>(lp, (unsigned)grid, st);
  return cudaGetLastError() == cudaSuccess ? PARARNN_OK : PARARNN_ERR_CUDA;
}
