// C ABI of the language-model operators: the head norms with rotation and the gated delta rule.
// Argument validation and launches; the operations, layouts and errors are documented in
// include/litela.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <utility>

#include "../../include/litela.h"
#include "litela_delta.cuh"
#include "litela_delta_bwd.cuh"
#include "litela_delta_chunk.cuh"
#include "litela_host.h"
#include "litela_norm.cuh"

namespace litela {

// set by a kernel whose bounded wait ran out (lite_la_device_status reads and clears it)
__device__ int g_delta_err;

int* delta_error_word(int) {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_delta_err) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  return static_cast<int*>(p);
}

namespace {

constexpr int kMaxTokens = 1 << 30;

litela_status invalid(const char* msg) { return host_fail(LITELA_ERR_INVALID_ARGUMENT, msg); }
litela_status unsupported(const char* msg) { return host_fail(LITELA_ERR_UNSUPPORTED, msg); }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// a span of device memory
struct Span {
  uintptr_t lo = 0, hi = 0;
};
Span span(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return p == nullptr || bytes == 0 ? Span{} : Span{a, a + bytes};
}
bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// launches `k` as a programmatic dependent of the previous kernel in the stream when `pdl`
template <typename... KArgs, typename... Args>
cudaError_t launch_seq(void (*k)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t stream, bool pdl,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k, static_cast<KArgs>(args)...);
}

// ---------------------------------------------------------------------------------------
// head norms with rotation

// The backward has two CTAs an SM: the workspace holds one pair of partial sums for each
constexpr int kNormMaxSms = 256, kNormMaxGrid = 2 * kNormMaxSms;

struct NormCall {
  const void *qkv, *dout;
  void* out;
  const float *wq, *wk, *cos, *sin;
  const void* pos;
  int pos_bytes, B, N, Hq, Hk, Hv, d, rot, table, inter;
  float eps;
};

litela_status norm_validate(const NormCall& c, bool bwd, bool* empty) {
  *empty = false;
  if (c.B < 0 || c.N < 0 || c.Hq < 0 || c.Hk < 0 || c.Hv < 0) return invalid("B, N, Hq, Hk and Hv must be >= 0");
  if (c.B > 65535 || c.N > kMaxTokens || c.Hq > 65535 || c.Hk > 65535 || c.Hv > 65535)
    return invalid("B and the heads must be <= 65535, N <= 2^30");
  if (c.d != 32 && c.d != 64 && c.d != 128) return unsupported("d must be 32, 64 or 128");
  if (c.rot < 0 || c.rot > c.d || c.rot % 16 != 0) return unsupported("rot must be a multiple of 16 up to d");
  if (!std::isfinite(c.eps) || c.eps < 0.f) return invalid("eps must be finite and >= 0");
  if (c.rot > 0 && c.table < 1) return invalid("the tables need at least one position");
  if (c.pos != nullptr && c.pos_bytes != 4 && c.pos_bytes != 8) return invalid("position_bytes must be 4 or 8");
  if (c.rot > 0 && c.pos == nullptr && c.table < c.N) return invalid("the tables are shorter than N");
  const double elems = (double)c.B * c.N * ((double)c.Hq + c.Hk + c.Hv) * c.d;
  if (elems > 4.0e18) return invalid("element count overflows int64");
  if (elems == 0) {
    *empty = true;
    return LITELA_OK;
  }
  if (c.qkv == nullptr || c.out == nullptr || (bwd && c.dout == nullptr)) return invalid("null buffer");
  if (c.rot > 0 && (c.cos == nullptr || c.sin == nullptr)) return invalid("null cos or sin");
  if (!aligned(c.qkv, 16) || !aligned(c.out, 16) || !aligned(c.dout, 16) || !aligned(c.cos, 16) || !aligned(c.sin, 16))
    return invalid("buffers and tables must be 16-byte aligned");
  if (!aligned(c.wq, 4) || !aligned(c.wk, 4) || !aligned(c.pos, c.pos ? c.pos_bytes : 1))
    return invalid("weights and positions must be aligned to their elements");
  const size_t n = (size_t)elems * 2;
  const Span o = span(c.out, n);
  const bool in_place = bwd ? c.out == c.dout : c.out == c.qkv;
  if ((bwd && meet(o, span(c.qkv, n))) || (!in_place && meet(o, span(bwd ? c.dout : c.qkv, n))))
    return invalid(bwd ? "dqkv overlaps qkv or dout" : "out overlaps qkv");
  const size_t tab = (size_t)c.table * (c.rot / 2) * 4;
  if (meet(o, span(c.wq, c.d * 4)) || meet(o, span(c.wk, c.d * 4)) || meet(o, span(c.cos, tab)) ||
      meet(o, span(c.sin, tab)) || meet(o, span(c.pos, (size_t)c.B * c.N * c.pos_bytes)))
    return invalid("the output overlaps a weight, a table or the positions");
  return LITELA_OK;
}

NormPlan norm_plan(const NormCall& c, bool bwd, int num_sms, int* grid) {
  NormPlan p{};
  p.x = static_cast<const __nv_bfloat16*>(c.qkv);
  p.dy = static_cast<const __nv_bfloat16*>(c.dout);
  p.out = static_cast<__nv_bfloat16*>(c.out);
  p.wq = c.wq, p.wk = c.wk, p.cos = c.cos, p.sin = c.sin, p.pos = c.pos;
  p.pos64 = c.pos_bytes == 8;
  p.rows = (long long)c.B * c.N;
  p.N = c.N;
  p.table = c.table;
  p.rot = c.rot;
  p.q_ch = c.Hq * c.d;
  p.qk_ch = (c.Hq + c.Hk) * c.d;
  p.W = p.qk_ch + c.Hv * c.d;
  p.copy_v = bwd ? c.out != c.dout : c.out != c.qkv;
  p.eps = c.eps;
  // padded rows of the backward are zeroed whole, v's part of an in-place one too
  p.regions = p.copy_v || (bwd && c.pos != nullptr) ? 3 : 2;
  // warps per task: enough to give every SM 16 warps, no more than a task has steps
  const long long tasks = p.rows * p.regions;
  const int widest = std::max(std::max(p.q_ch, p.qk_ch - p.q_ch), p.regions == 3 ? p.W - p.qk_ch : 0);
  while ((tasks << p.shift) < 16LL * num_sms && (kNormStep << p.shift) < widest) ++p.shift;
  const long long ctas = ((tasks << p.shift) + kNormWarps - 1) / kNormWarps;
  *grid = (int)std::min<long long>(ctas, (bwd ? 2 : 3) * std::min(num_sms, kNormMaxSms));   // as many as fit at once
  return p;
}

template <bool kBwd>
cudaError_t norm_launch(const NormPlan& p, int d, bool inter, int grid, cudaStream_t st) {
#define LITELA_NORM(D, I)                                                                             \
  return kBwd ? launch_seq(litela_norm_bwd<D, I>, dim3(grid), kNormThreads, 0, st, false, p)          \
              : launch_seq(litela_norm_fwd<D, I>, dim3(grid), kNormThreads, 0, st, false, p)
  if (d == 32) {
    if (inter) LITELA_NORM(32, true);
    LITELA_NORM(32, false);
  }
  if (d == 64) {
    if (inter) LITELA_NORM(64, true);
    LITELA_NORM(64, false);
  }
  if (inter) LITELA_NORM(128, true);
  LITELA_NORM(128, false);
#undef LITELA_NORM
}

litela_status norm_fwd(const NormCall& c, cudaStream_t st) {
  bool empty;
  litela_status s = norm_validate(c, false, &empty);
  if (s != LITELA_OK || empty) return s;
  int dev, sms, grid;
  if ((s = host_device(&dev, &sms)) != LITELA_OK) return s;
  const NormPlan p = norm_plan(c, false, sms, &grid);
  if (p.qk_ch == 0 && !p.copy_v) return LITELA_OK;
  const cudaError_t e = norm_launch<false>(p, c.d, c.inter != 0, grid, st);
  if (e != cudaSuccess) return host_cuda_fail(e, "launch litela_norm_fwd");
  host_ok();
  return LITELA_OK;
}

litela_status norm_bwd(const NormCall& c, float* dwq, float* dwk, void* ws, size_t ws_bytes, cudaStream_t st) {
  bool empty;
  litela_status s = norm_validate(c, true, &empty);
  if (s != LITELA_OK) return s;
  if (!aligned(dwq, 4) || !aligned(dwk, 4)) return invalid("the weights' gradients must be 4-byte aligned");
  const bool weights = dwq != nullptr || dwk != nullptr;
  const size_t n = (size_t)c.B * c.N * ((size_t)c.Hq + c.Hk + c.Hv) * c.d * 2;
  const size_t need = lite_la_qk_norm_rope_workspace_bytes(c.d);
  if (weights && !empty) {
    if (ws == nullptr || ws_bytes < need || !aligned(ws, 16)) return invalid("workspace missing, too small or misaligned");
    const Span w = span(ws, ws_bytes), outs[3] = {span(c.out, n), span(dwq, c.d * 4), span(dwk, c.d * 4)};
    for (const Span& o : outs)
      if (meet(w, o)) return invalid("the workspace overlaps an output");
    if (meet(w, span(c.qkv, n)) || meet(w, span(c.dout, n))) return invalid("the workspace overlaps an input");
    if (meet(outs[0], outs[1]) || meet(outs[0], outs[2]) || meet(outs[1], outs[2])) return invalid("outputs overlap");
    for (int i = 1; i < 3; ++i)
      if (meet(outs[i], span(c.qkv, n)) || meet(outs[i], span(c.dout, n)) || meet(outs[i], span(c.wq, c.d * 4)) ||
          meet(outs[i], span(c.wk, c.d * 4)))
        return invalid("a weight's gradient overlaps an input");
  }
  int dev, sms, grid;
  if ((s = host_device(&dev, &sms)) != LITELA_OK) return s;
  if (empty) {   // no rows: the weights' gradients are zero
    for (float* w : {dwq, dwk})
      if (w != nullptr) {
        const cudaError_t e = cudaMemsetAsync(w, 0, c.d * sizeof(float), st);
        if (e != cudaSuccess) return host_cuda_fail(e, "cudaMemsetAsync");
      }
    return LITELA_OK;
  }
  NormPlan p = norm_plan(c, true, sms, &grid);
  p.partials = weights ? static_cast<float*>(ws) : nullptr;
  cudaError_t e = norm_launch<true>(p, c.d, c.inter != 0, grid, st);
  if (e != cudaSuccess) return host_cuda_fail(e, "launch litela_norm_bwd");
  if (weights) {
    e = launch_seq(litela_norm_weight_grad, dim3(2 * c.d), 32, 0, st, true, static_cast<const float*>(p.partials), grid,
                   c.d, dwq, dwk);
    if (e != cudaSuccess) return host_cuda_fail(e, "launch litela_norm_weight_grad");
  }
  host_ok();
  return LITELA_OK;
}

// ---------------------------------------------------------------------------------------
// the gated delta rule

// checks a view of [B, N, heads, d]; `out`: no two of its rows may share memory
litela_status view_check(const lite_la_view& v, int B, int N, int heads, int d, bool out, Span* sp) {
  *sp = Span{};
  if (B == 0 || N == 0 || heads == 0) return LITELA_OK;
  if (v.data == nullptr) return invalid("null q, k, v, out or gradient");
  if (!aligned(v.data, 16)) return invalid("views must be 16-byte aligned");
  const struct { long long stride; int size; } dim[3] = {
      {v.batch_stride, B}, {v.token_stride, N}, {v.head_stride, heads}};
  double last = d;
  for (const auto& x : dim) {
    if (x.size == 1) continue;
    if (x.stride < 0 || x.stride % 8 != 0) return invalid("view strides must be multiples of 8 and >= 0");
    last += (double)x.stride * (x.size - 1);
  }
  if (last > 4.0e18) return invalid("a view's extent overflows int64");
  if (out) {   // sorted by stride, each dimension has to step over all of the smaller ones
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return dim[a].stride < dim[b].stride; });
    double extent = d;
    for (int i : order) {
      if (dim[i].size == 1) continue;
      if ((double)dim[i].stride < extent) return invalid("an output view overlaps itself");
      extent += (double)dim[i].stride * (dim[i].size - 1);
    }
  }
  *sp = span(v.data, (size_t)last * 2);
  return LITELA_OK;
}

size_t gate_bytes(int B, int N, int H, long long sb, long long st) {
  return B == 0 || N == 0 || H == 0 ? 0 : ((size_t)(B - 1) * sb + (size_t)(N - 1) * st + H) * 4;
}

// inputs' spans of a call, for the outputs to keep clear of
struct DeltaSpans {
  Span in[8];
  int n = 0;
  void add(const Span& s) { in[n++] = s; }
  bool hit(const Span& o) const {
    for (int i = 0; i < n; ++i)
      if (meet(in[i], o)) return true;
    return false;
  }
};

// host-side checks shared by the gated delta rule's calls; *empty: no sequences or no heads
litela_status delta_validate(const lite_la_delta_args* a, bool with_out, DeltaSpans* in, Span* out, bool* empty) {
  *empty = false;
  if (a == nullptr) return invalid("null args");
  if (a->B < 0 || a->N < 0 || a->Hk < 0 || a->Hv < 0) return invalid("B, N, Hk and Hv must be >= 0");
  if (a->B > 65535 || a->Hv > 65535 || a->Hk > 65535 || a->N > kMaxTokens)
    return invalid("B and the heads must be <= 65535, N <= 2^30");
  if (a->d != 32 && a->d != 64 && a->d != 128) return unsupported("d must be 32, 64 or 128");
  if ((a->Hk == 0) != (a->Hv == 0) || (a->Hk > 0 && a->Hv % a->Hk != 0))
    return unsupported("Hv must be a multiple of Hk");
  if (!std::isfinite(a->scale)) return invalid("scale must be finite");
  if (a->cu_seqlens != nullptr && a->B == 0 && a->N > 0) return invalid("packed tokens need a sequence");
  if (a->B == 0 || a->Hv == 0) {
    *empty = true;
    return LITELA_OK;
  }
  if ((double)a->B * a->Hv * (a->d / 32) > 2147483647.0) return invalid("too many sequences and heads");
  const int entries = a->cu_seqlens != nullptr ? 1 : a->B;
  Span s;
  litela_status st;
  if ((st = view_check(a->q, entries, a->N, a->Hk, a->d, false, &s)) != LITELA_OK) return st;
  in->add(s);
  if ((st = view_check(a->k, entries, a->N, a->Hk, a->d, false, &s)) != LITELA_OK) return st;
  in->add(s);
  if ((st = view_check(a->v, entries, a->N, a->Hv, a->d, false, &s)) != LITELA_OK) return st;
  in->add(s);
  if (a->N > 0) {
    if (a->g == nullptr || a->beta == nullptr) return invalid("null g or beta");
    if (!aligned(a->g, 4) || !aligned(a->beta, 4)) return invalid("g and beta must be 4-byte aligned");
    if (a->g_batch_stride < 0 || a->g_token_stride < 0 || a->beta_batch_stride < 0 || a->beta_token_stride < 0)
      return invalid("strides of g and beta must be >= 0");
    for (const auto& x : {std::pair<long long, long long>(a->g_batch_stride, a->g_token_stride),
                          std::pair<long long, long long>(a->beta_batch_stride, a->beta_token_stride)})
      if ((double)x.first * entries + (double)x.second * a->N > 2.0e18) return invalid("a gate's extent overflows int64");
    in->add(span(a->g, gate_bytes(entries, a->N, a->Hv, a->g_batch_stride, a->g_token_stride)));
    in->add(span(a->beta, gate_bytes(entries, a->N, a->Hv, a->beta_batch_stride, a->beta_token_stride)));
  }
  if (!aligned(a->state_in, 16) || !aligned(a->state_out, 16)) return invalid("states must be 16-byte aligned");
  if (!aligned(a->cu_seqlens, 4)) return invalid("cu_seqlens must be 4-byte aligned");
  in->add(span(a->cu_seqlens, a->cu_seqlens ? ((size_t)a->B + 1) * 4 : 0));
  if (with_out) {
    if ((st = view_check(a->out, entries, a->N, a->Hv, a->d, true, out)) != LITELA_OK) return st;
    if (in->hit(*out)) return invalid("out overlaps an input");
  }
  return LITELA_OK;
}

litela_status state_check(const lite_la_delta_args* a, size_t bytes, const DeltaSpans& in, const Span& out) {
  const Span si = span(a->state_in, bytes), so = span(a->state_out, bytes);
  if (meet(si, out) || meet(so, out)) return invalid("a state overlaps out");
  if (in.hit(so)) return invalid("state_out overlaps an input");
  if (a->state_in != a->state_out && meet(si, so)) return invalid("state_out overlaps state_in in part");
  return LITELA_OK;
}

DeltaView view_of(const lite_la_view& v) {
  return DeltaView{static_cast<__nv_bfloat16*>(v.data), v.batch_stride, v.token_stride, v.head_stride};
}

DeltaArgs delta_args(const lite_la_delta_args* a) {
  DeltaArgs d{};
  d.q = view_of(a->q), d.k = view_of(a->k), d.v = view_of(a->v), d.out = view_of(a->out);
  d.g = a->g, d.beta = a->beta;
  d.g_sb = a->g_batch_stride, d.g_st = a->g_token_stride;
  d.b_sb = a->beta_batch_stride, d.b_st = a->beta_token_stride;
  d.state_in = a->state_in, d.state_out = a->state_out;
  d.cu = a->cu_seqlens;
  d.nseq = a->B, d.ntok = a->N, d.Hk = a->Hk, d.Hv = a->Hv;
  d.scale = a->scale;
  return d;
}

litela_status launch_recur(const DeltaArgs& d, int D, cudaStream_t st) {
  const dim3 grid((unsigned)((long long)d.nseq * d.Hv * (D / kRecurCols)));
  const bool one = d.cu == nullptr && d.ntok == 1;
#define LITELA_RECUR(D)                                                            \
  (one ? launch_seq(litela_delta_step<D>, grid, kRecurThreads, 0, st, false, d)    \
       : launch_seq(litela_delta_recur<D>, grid, kRecurThreads, 0, st, false, d))
  const cudaError_t e = D == 32 ? LITELA_RECUR(32) : D == 64 ? LITELA_RECUR(64) : LITELA_RECUR(128);
#undef LITELA_RECUR
  return e == cudaSuccess ? LITELA_OK : host_cuda_fail(e, "launch the recurrence");
}

// shared-memory limits of the chunked kernels, once per device
litela_status delta_setup(int dev) {
  static std::mutex mutex;
  static bool ready[64] = {};
  std::lock_guard<std::mutex> lock(mutex);
  if (ready[dev]) return LITELA_OK;
  cudaError_t e = cudaSuccess;
  auto set = [&](auto* k, uint32_t bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  };
  set(litela_delta_prep<32, false>, PrepCfg<32>::kSmemBytes);
  set(litela_delta_prep<64, false>, PrepCfg<64>::kSmemBytes);
  set(litela_delta_prep<128, false>, PrepCfg<128>::kSmemBytes);
  set(litela_delta_prep<32, true>, PrepCfg<32>::kSmemBytes);
  set(litela_delta_prep<64, true>, PrepCfg<64>::kSmemBytes);
  set(litela_delta_prep<128, true>, PrepCfg<128>::kSmemBytes);
  set(litela_delta_chain<32, false>, ChainCfg<32>::kSmemBytes);
  set(litela_delta_chain<64, false>, ChainCfg<64>::kSmemBytes);
  set(litela_delta_chain<128, false>, ChainCfg<128>::kSmemBytes);
  set(litela_delta_chain<32, true>, ChainCfg<32>::kSmemBytes);
  set(litela_delta_chain<64, true>, ChainCfg<64>::kSmemBytes);
  set(litela_delta_chain<128, true>, ChainCfg<128>::kSmemBytes);
  set(litela_delta_back<32>, BackCfg<32>::kSmemBytes);
  set(litela_delta_back<64>, BackCfg<64>::kSmemBytes);
  set(litela_delta_back<128>, BackCfg<128>::kSmemBytes);
  set(litela_delta_grads<32>, GradCfg<32>::kSmemBytes);
  set(litela_delta_grads<64>, GradCfg<64>::kSmemBytes);
  set(litela_delta_grads<128>, GradCfg<128>::kSmemBytes);
  if (e != cudaSuccess) return host_cuda_fail(e, "cudaFuncSetAttribute(dynamic shared memory)");
  ready[dev] = true;
  return LITELA_OK;
}

// The recurrence or the chunks.  The recurrence takes 0.20 to 0.25 us a token (one sequence, d = 32
// to 128) or what its instructions take; the chunks take a whole chunk's time for every started one.  Dense
// (us in a graph, recurrence / chunks), N = 32: 1 x 32 heads of 128 12 / 17, 64 x 32 291 / 381; 1 x 8 heads of 64
// 10 / 14, 64 x 8 30 / 55; 1 x 70 heads of 32 10 / 14, 64 x 70 83 / 274.  N = 48: 17 / 17, 424 / 385,
// 14 / 14, 42 / 56, 14 / 14, 121 / 277.  N = 64: 21 / 17, 557 / 392, 19 / 14, 54 / 56, 17 / 14, 158 / 280.
// Packed lengths are known to the device only, and all tokens may be one sequence's: the recurrence where
// they are 8 on the average and no sequence can have more than 512 (the same heads: 64 sequences of 8
// 105 / 385, 12 / 56, 29 / 271; one of 512 and 63 without tokens 295 / 201, 119 / 45, 128 / 105).  The rule
// guards the second kind and gives up some of the first: 16 sequences of 12 take 107, 21 and 72 as chunks
// where the recurrence would take 39, 8 and 12; 128 of 5 762, 103 and 519 where it would take 174, 18 and 44.
constexpr int kRecurMaxTokens = 32, kRecurMaxMean = 8, kRecurMaxPacked = 512;
bool delta_recurs(int nseq, int ntok, bool packed) {
  if (ntok <= kRecurMaxTokens) return true;
  return packed && ntok <= kRecurMaxPacked && ntok <= (long long)kRecurMaxMean * nseq;
}

// the prepared blocks, then the chain; kSave: a training step's
template <int kD, bool kSave = false>
cudaError_t launch_chunks(const DeltaArgs& d, uint8_t* prep, int* err, cudaStream_t st, DeltaSaved saved = {}) {
  const long long slots = delta_slots(d.nseq, d.ntok, d.cu != nullptr);
  const cudaError_t e = launch_seq(litela_delta_prep<kD, kSave>, dim3((unsigned)(slots * d.Hv)), kPrepThreads,
                                   PrepCfg<kD>::kSmemBytes, st, false, d, prep);
  if (e != cudaSuccess) return e;
  return launch_seq(litela_delta_chain<kD, kSave>, dim3((unsigned)((long long)d.nseq * d.Hv * (kD / kCols))), kChainThreads,
                    ChainCfg<kD>::kSmemBytes, st, true, d, static_cast<const uint8_t*>(prep), saved, err);
}

// bytes of a call's buffers per chunk slot and value head, and their places
struct DeltaBytes {
  size_t n;   // slots x value heads
  size_t prep, kept, states, gstates, rows, shares, ends;
  explicit DeltaBytes(const DeltaArgs& d, int D) : DeltaBytes(d.nseq, d.ntok, d.Hv, D, d.cu != nullptr) {}
  DeltaBytes(int B, int N, int Hv, int D, bool packed)
      : n(N > 0 ? (size_t)delta_slots(B, N, packed) * Hv : 0),   // (packed: there are slots without tokens)
        prep(up(n * kPrepBytes)),
        kept(up(n * kPrepSaveBytes)),
        states(up(n * D * D * 8)),
        gstates(up(n * D * D * 4)),
        rows(up(n * kChunk * D * 4)),
        shares(up(n * (D / 32) * 4 * kChunk * 4)),
        ends(up(n * (D / 32) * 8 * 4)) {}
  static size_t up(size_t x) { return (x + 255) / 256 * 256; }
  size_t saved() const { return kept + states + rows; }
  size_t back() const { return gstates + rows + shares + ends; }
};

bool delta_sizes_ok(int B, int N, int Hk, int Hv, int d) {
  return B > 0 && N > 0 && Hk > 0 && Hv > 0 && (d == 32 || d == 64 || d == 128);
}

DeltaSaved delta_saved(const DeltaBytes& b, void* saved) {
  uint8_t* p = static_cast<uint8_t*>(saved);
  return DeltaSaved{p + b.kept, reinterpret_cast<float*>(p + b.kept + b.states)};
}

template <int kD>
cudaError_t launch_save(const DeltaArgs& d, void* saved, int* err, cudaStream_t st) {
  return launch_chunks<kD, true>(d, static_cast<uint8_t*>(saved), err, st, delta_saved(DeltaBytes(d, kD), saved));
}

template <int kD>
cudaError_t launch_back(const DeltaArgs& d, const DeltaGrads& g, const void* saved, int* err, cudaStream_t st) {
  const uint8_t* prep = static_cast<const uint8_t*>(saved);
  const DeltaSaved kept = delta_saved(DeltaBytes(d, kD), const_cast<void*>(saved));
  cudaError_t e = launch_seq(litela_delta_back<kD>, dim3((unsigned)((long long)d.nseq * d.Hv * (kD / 32))), kChainThreads,
                             BackCfg<kD>::kSmemBytes, st, false, d, g, prep, kept, err);
  if (e != cudaSuccess || d.ntok == 0) return e;
  const long long slots = delta_slots(d.nseq, d.ntok, d.cu != nullptr);
  return launch_seq(litela_delta_grads<kD>, dim3((unsigned)(slots * d.Hk)), GradCfg<kD>::kThreads, GradCfg<kD>::kSmemBytes, st, true,
                    d, g, prep, kept);
}

// a call's workspace or kept data: present, aligned and clear of the call's other buffers
litela_status buffer_check(const lite_la_delta_args* a, const void* p, size_t bytes, size_t need, const DeltaSpans& in,
                           const Span& out, const char* missing, const char* overlap) {
  if (need > 0 && (p == nullptr || bytes < need || !aligned(p, 16))) return invalid(missing);
  const Span w = span(p, need);
  const size_t states = (size_t)a->B * a->Hv * a->d * a->d * 4;
  if (meet(w, out) || in.hit(w) || meet(w, span(a->state_in, states)) || meet(w, span(a->state_out, states)))
    return invalid(overlap);
  if (delta_slots(a->B, a->N, a->cu_seqlens != nullptr) * (double)a->Hv > 2147483647.0)
    return invalid("too many chunks and heads");
  return LITELA_OK;
}

litela_status delta_fwd(const lite_la_delta_args* a, bool save, void* saved, size_t saved_bytes, cudaStream_t st) {
  DeltaSpans in;
  Span out;
  bool empty;
  litela_status s = delta_validate(a, true, &in, &out, &empty);
  if (s != LITELA_OK || empty) return s;
  if ((s = state_check(a, (size_t)a->B * a->Hv * a->d * a->d * 4, in, out)) != LITELA_OK) return s;
  const bool recurs = !save && delta_recurs(a->B, a->N, a->cu_seqlens != nullptr);
  const DeltaBytes bytes(a->B, a->N, a->Hv, a->d, a->cu_seqlens != nullptr);
  if (save) {
    s = buffer_check(a, saved, saved_bytes, bytes.saved(), in, out, "saved missing, too small or misaligned",
                     "saved overlaps a buffer of the call");
  } else if (!recurs) {
    s = buffer_check(a, a->workspace, a->workspace_bytes, bytes.prep, in, out, "workspace missing, too small or misaligned",
                     "the workspace overlaps a buffer of the call");
  }
  if (s != LITELA_OK) return s;
  int dev, sms;
  if ((s = host_device(&dev, &sms)) != LITELA_OK) return s;
  DeltaArgs d = delta_args(a);
  d.zero_rest = a->zero_tail != 0 && a->cu_seqlens != nullptr;
  if (save) {
    if ((s = delta_setup(dev)) != LITELA_OK) return s;
    if (d.ntok == 0) {
      s = launch_recur(d, a->d, st);   // the states alone
    } else {
      int* err = delta_error_word(dev);
      const cudaError_t e = a->d == 32   ? launch_save<32>(d, saved, err, st)
                            : a->d == 64 ? launch_save<64>(d, saved, err, st)
                                         : launch_save<128>(d, saved, err, st);
      if (e != cudaSuccess) return host_cuda_fail(e, "launch the forward of a training step");
    }
  } else {
    if (recurs) {
      s = launch_recur(d, a->d, st);
    } else if ((s = delta_setup(dev)) == LITELA_OK) {
      uint8_t* ws = static_cast<uint8_t*>(a->workspace);
      int* err = delta_error_word(dev);
      const cudaError_t e = a->d == 32   ? launch_chunks<32>(d, ws, err, st)
                            : a->d == 64 ? launch_chunks<64>(d, ws, err, st)
                                         : launch_chunks<128>(d, ws, err, st);
      if (e != cudaSuccess) return host_cuda_fail(e, "launch the gated delta rule's chunks");
    }
  }
  if (s == LITELA_OK) host_ok();
  return s;
}

litela_status delta_bwd(const lite_la_delta_args* a, const lite_la_delta_grads* g, const void* saved, size_t saved_bytes,
                        cudaStream_t st) {
  if (g == nullptr) return invalid("null grads");
  DeltaSpans in;
  Span out, sp[3];
  bool empty;
  litela_status s = delta_validate(a, false, &in, &out, &empty);
  if (s != LITELA_OK || empty) return s;
  const int entries = a->cu_seqlens != nullptr ? 1 : a->B;
  Span dout;
  if ((s = view_check(g->dout, entries, a->N, a->Hv, a->d, false, &dout)) != LITELA_OK) return s;
  in.add(dout);
  if ((s = view_check(g->dq, entries, a->N, a->Hk, a->d, true, &sp[0])) != LITELA_OK ||
      (s = view_check(g->dk, entries, a->N, a->Hk, a->d, true, &sp[1])) != LITELA_OK ||
      (s = view_check(g->dv, entries, a->N, a->Hv, a->d, true, &sp[2])) != LITELA_OK)
    return s;
  if (a->N > 0 && (g->dg == nullptr || g->dbeta == nullptr)) return invalid("null dg or dbeta");
  if (!aligned(g->dg, 4) || !aligned(g->dbeta, 4)) return invalid("dg and dbeta must be 4-byte aligned");
  if (!aligned(g->dstate_out, 16) || !aligned(g->dstate_in, 16))
    return invalid("the states' gradients must be 16-byte aligned");
  const DeltaBytes bytes(a->B, a->N, a->Hv, a->d, a->cu_seqlens != nullptr);
  const size_t states = (size_t)a->B * a->Hv * a->d * a->d * 4, gates = (size_t)entries * a->N * a->Hv * 4;
  if ((s = buffer_check(a, saved, saved_bytes, bytes.saved(), in, Span{}, "saved missing, too small or misaligned",
                        "saved overlaps a buffer of the call")) != LITELA_OK ||
      (s = buffer_check(a, a->workspace, a->workspace_bytes, bytes.back(), in, Span{},
                        "workspace missing, too small or misaligned", "the workspace overlaps a buffer of the call")) !=
          LITELA_OK)
    return s;
  in.add(span(saved, bytes.saved()));
  const Span dso = span(g->dstate_out, states);
  // dq, dk, dv may be views of one buffer between one another's rows: only their spans against inputs
  // and the dense outputs are checked
  const Span outs[7] = {sp[0], sp[1], sp[2], span(g->dg, gates), span(g->dbeta, gates), span(g->dstate_in, states),
                        span(a->workspace, bytes.back())};
  for (int i = 0; i < 3; ++i)
    if (sp[i].hi > 0 && sp[i].lo == sp[(i + 1) % 3].lo) return invalid("dq, dk and dv must be different memory");
  for (int i = 0; i < 7; ++i) {
    if (in.hit(outs[i]) || (i != 5 && meet(outs[i], dso))) return invalid("an output overlaps an input");
    for (int j = i + 1; j < 7; ++j)
      if (j > 2 && meet(outs[i], outs[j])) return invalid("outputs overlap");
  }
  if (g->dstate_in != nullptr && g->dstate_in != g->dstate_out && meet(outs[5], dso))
    return invalid("dstate_in overlaps dstate_out in part");
  int dev, sms;
  if ((s = host_device(&dev, &sms)) != LITELA_OK || (s = delta_setup(dev)) != LITELA_OK) return s;
  DeltaArgs d = delta_args(a);
  d.zero_rest = a->cu_seqlens != nullptr;
  DeltaGrads gr{};
  gr.dout = view_of(g->dout), gr.dq = view_of(g->dq), gr.dk = view_of(g->dk), gr.dv = view_of(g->dv);
  gr.dg = g->dg, gr.dbeta = g->dbeta;
  gr.dstate_out = g->dstate_out, gr.dstate_in = g->dstate_in;
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  gr.gstates = ws;
  gr.y = reinterpret_cast<float*>(ws + bytes.gstates);
  gr.rows = reinterpret_cast<float*>(ws + bytes.gstates + bytes.rows);
  gr.ends = reinterpret_cast<float*>(ws + bytes.gstates + bytes.rows + bytes.shares);
  int* err = delta_error_word(dev);
  const cudaError_t e = a->d == 32   ? launch_back<32>(d, gr, saved, err, st)
                        : a->d == 64 ? launch_back<64>(d, gr, saved, err, st)
                                     : launch_back<128>(d, gr, saved, err, st);
  if (e != cudaSuccess) return host_cuda_fail(e, "launch the gated delta rule's gradient");
  host_ok();
  return LITELA_OK;
}

litela_status delta_step(const lite_la_delta_args* a, const int* slots, int pool, cudaStream_t st) {
  DeltaSpans in;
  Span out;
  bool empty;
  litela_status s = delta_validate(a, true, &in, &out, &empty);
  if (s != LITELA_OK) return s;
  if (pool < 0) return invalid("pool must be >= 0");
  if (a->cu_seqlens != nullptr) return invalid("the one-token form takes no cu_seqlens");
  if (empty) return LITELA_OK;
  if (a->N != 1) return invalid("the one-token form needs N = 1");
  if (a->state_in != a->state_out || a->state_in == nullptr)
    if (pool > 0 || a->state_in != a->state_out) return invalid("state_in and state_out must be the same pool");
  if (slots == nullptr && pool < a->B) return invalid("the pool has fewer states than the batch has rows");
  if (!aligned(slots, 4)) return invalid("state_indices must be 4-byte aligned");
  in.add(span(slots, slots ? (size_t)a->B * 4 : 0));
  if (in.hit(out)) return invalid("out overlaps an input");
  if ((s = state_check(a, (size_t)pool * a->Hv * a->d * a->d * 4, in, out)) != LITELA_OK) return s;
  int dev, sms;
  if ((s = host_device(&dev, &sms)) != LITELA_OK) return s;
  DeltaArgs d = delta_args(a);
  d.slots = slots;
  d.nslots = pool;
  if ((s = launch_recur(d, a->d, st)) != LITELA_OK) return s;
  host_ok();
  return LITELA_OK;
}

// no C++ exception leaves a C entry point
template <typename F>
litela_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return LITELA_ERR_OUT_OF_MEMORY;
  }
}

}  // namespace
}  // namespace litela

extern "C" {

litela_status lite_la_qk_norm_rope_fwd(const void* qkv, void* out, const float* q_weight, const float* k_weight,
                                       const float* cos, const float* sin, const void* positions, int position_bytes,
                                       int B, int N, int Hq, int Hk, int Hv, int d, int rot, int table_len,
                                       int interleaved, float eps, cudaStream_t stream) {
  return litela::guarded([&] {
    return litela::norm_fwd({qkv, nullptr, out, q_weight, k_weight, cos, sin, positions, position_bytes, B, N, Hq, Hk,
                             Hv, d, rot, table_len, interleaved, eps},
                            stream);
  });
}

litela_status lite_la_qk_norm_rope_bwd(const void* qkv, const void* dout, void* dqkv, const float* q_weight,
                                       const float* k_weight, float* dq_weight, float* dk_weight, const float* cos,
                                       const float* sin, const void* positions, int position_bytes, int B, int N,
                                       int Hq, int Hk, int Hv, int d, int rot, int table_len, int interleaved,
                                       float eps, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return litela::guarded([&] {
    return litela::norm_bwd({qkv, dout, dqkv, q_weight, k_weight, cos, sin, positions, position_bytes, B, N, Hq, Hk, Hv,
                             d, rot, table_len, interleaved, eps},
                            dq_weight, dk_weight, workspace, workspace_bytes, stream);
  });
}

size_t lite_la_qk_norm_rope_workspace_bytes(int d) {
  return d == 32 || d == 64 || d == 128 ? (size_t)litela::kNormMaxGrid * 2 * d * sizeof(float) : 0;
}

litela_status lite_la_gated_delta_fwd(const lite_la_delta_args* args, cudaStream_t stream) {
  return litela::guarded([&] { return litela::delta_fwd(args, false, nullptr, 0, stream); });
}

size_t lite_la_gated_delta_workspace_bytes(int B, int N, int Hk, int Hv, int d, int packed) {
  if (!litela::delta_sizes_ok(B, N, Hk, Hv, d) || litela::delta_recurs(B, N, packed != 0)) return 0;
  return litela::DeltaBytes(B, N, Hv, d, packed != 0).prep;
}

litela_status lite_la_gated_delta_fwd_save(const lite_la_delta_args* args, void* saved, size_t saved_bytes,
                                           cudaStream_t stream) {
  return litela::guarded([&] { return litela::delta_fwd(args, true, saved, saved_bytes, stream); });
}

size_t lite_la_gated_delta_saved_bytes(int B, int N, int Hk, int Hv, int d, int packed) {
  return litela::delta_sizes_ok(B, N, Hk, Hv, d) ? litela::DeltaBytes(B, N, Hv, d, packed != 0).saved() : 0;
}

litela_status lite_la_gated_delta_bwd(const lite_la_delta_args* args, const lite_la_delta_grads* grads,
                                      const void* saved, size_t saved_bytes, cudaStream_t stream) {
  return litela::guarded([&] { return litela::delta_bwd(args, grads, saved, saved_bytes, stream); });
}

size_t lite_la_gated_delta_bwd_workspace_bytes(int B, int N, int Hk, int Hv, int d, int packed) {
  return litela::delta_sizes_ok(B, N, Hk, Hv, d) ? litela::DeltaBytes(B, N, Hv, d, packed != 0).back() : 0;
}

litela_status lite_la_gated_delta_step(const lite_la_delta_args* args, const int* state_indices, int pool,
                                       cudaStream_t stream) {
  return litela::guarded([&] { return litela::delta_step(args, state_indices, pool, stream); });
}

}  // extern "C"
