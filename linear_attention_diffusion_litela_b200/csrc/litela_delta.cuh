// The gated delta rule: arguments shared by its kernels, and the recurrent kernel.
//
// Per sequence and value head (key head = value head / group), with q, k the key head's d
// channels, v the value head's, g the log decay and beta the write strength of a token, and a
// d x d state S (rows: key channels, columns: value channels):
//     S <- e^g S + k (beta (v - e^g S^T k))^T,     out = scale * S^T q.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "f32x2.cuh"
#include "sm100_ptx.cuh"

namespace litela {

// a bf16 [entry, token, head, d] operand: strides in elements, the d channels of a head adjacent
struct DeltaView {
  __nv_bfloat16* p;
  long long sb, st, sh;
};

struct DeltaArgs {
  DeltaView q, k, v, out;
  const float* g;              // [entry, token, head], head stride 1
  const float* beta;
  long long g_sb, g_st, b_sb, b_st;
  const float* state_in;       // [sequence or slot][Hv][d][d], or null (zeros)
  float* state_out;            // may be state_in, or null
  const int* cu;               // packed: first token of each sequence, nseq + 1 entries; else null
  const int* slots;            // state of sequence s is slots[s] (both state_in and state_out); else null
  int nseq;                    // sequences (batch entries when not packed)
  int ntok;                    // tokens: of the packed buffer, or of each batch entry
  int nslots;                  // states in the pool (slots != null)
  int Hk, Hv;
  int zero_rest;               // packed: rows of no sequence are set to zero
  float scale;
};

// A log decay below this decays to zero in fp32 (e^-110 is under half the smallest subnormal);
// -inf and anything as low count as this, so that sums of decays stay finite.
constexpr float kMinLogDecay = -110.f;
__device__ __forceinline__ float clamp_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }

// Sequence s: its batch entry (packed: 0) and its tokens [first, first + len) there.  The packed
// offsets are device data: whatever they hold, the tokens stay inside the buffer.
struct DeltaSeq {
  int entry, first, len;
};
__device__ __forceinline__ DeltaSeq delta_seq(const DeltaArgs& a, int s) {
  if (a.cu == nullptr) return DeltaSeq{s, 0, a.ntok};
  const int b = min(max(a.cu[s], 0), a.ntok), e = min(max(a.cu[s + 1], b), a.ntok);
  return DeltaSeq{0, b, e - b};
}

__device__ __forceinline__ const __nv_bfloat16* delta_row(const DeltaView& v, const DeltaSeq& s, int n, int h) {
  return v.p + s.entry * v.sb + (long long)(s.first + n) * v.st + h * v.sh;
}

__device__ __forceinline__ float bf16_up(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// Rows of a packed buffer that no sequence has (those before the first one and behind the last one):
// this thread's share of the grid's.  f(row, one of its per_row pieces)
template <typename F>
__device__ __forceinline__ void delta_rest(const DeltaArgs& a, int per_row, F&& f) {
  const int b = min(max(a.cu[0], 0), a.ntok), e = min(max(a.cu[a.nseq], b), a.ntok);
  const long long n = (long long)(b + a.ntok - e) * per_row;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const int row = (int)(i / per_row);
    f(row < b ? row : e + row - b, (int)(i - (long long)row * per_row));
  }
}
// zeros there, in an output of `heads` heads of d channels
__device__ __forceinline__ void delta_zero_rest(const DeltaArgs& a, const DeltaView& out, int heads, int d) {
  delta_rest(a, heads * (d / 8), [&](int row, int c) {
    *reinterpret_cast<uint4*>(out.p + (long long)row * out.st + (c / (d / 8)) * out.sh + (c % (d / 8)) * 8) =
        make_uint4(0u, 0u, 0u, 0u);
  });
}

// ---------------------------------------------------------------------------------------
// litela_delta_recur: the recurrence, one token after another, the state in registers.
//
// A warp owns 8 columns of one state (all d rows): lane = d / 16 rows (of group lane / 2) and 4
// columns (of half lane & 1).  Nothing is shared between warps.  Two tokens are taken at a time: the
// products of the state before them with both k and both q are summed in the same shuffles (each
// halves the sums that a lane still holds, until it has one of the 16 totals of its columns), and
// with a, b the tokens' decays e^g and beta, S that state,
//     u1 = b1 (v1 - a1 S^T k1),    u2 = b2 (v2 - a2 (a1 S^T k2 + (k1 . k2) u1)),
//     out1 = scale (a1 S^T q1 + (k1 . q1) u1),
//     out2 = scale (a1 a2 S^T q2 + a2 (k1 . q2) u1 + (k2 . q2) u2),    S <- a1 a2 S + a2 k1 u1^T + k2 u2^T.
// Tokens come through shared memory, kRecurBatch at a time while the batch before is worked on.  Bound by
// the chain of dependent sums, 0.20 us a token (d = 32) to 0.25 us (128); one token at a time took 0.26 to 0.4.
// 16 sequences of 125 tokens in all, the longest of 30, 8 heads of 64: 12 us (15 by single tokens; 23
// with each token loaded from global memory one ahead).  The grid is one CTA per 32 columns, so that one
// sequence already fills the SMs.
constexpr int kRecurThreads = 128;
constexpr int kRecurCols = 32;
constexpr int kRecurBatch = 8;

// kN bf16 values, kN / 2 words
template <int kN>
__device__ __forceinline__ void recur_load(const uint8_t* p, uint32_t* w) {
  if (kN == 8) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if (kN == 4) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    w[0] = x.x, w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

template <int kD>
__global__ void __launch_bounds__(kRecurThreads) litela_delta_recur(const DeltaArgs a) {
  using namespace sm100;
  constexpr int kRows = kD / 16;   // rows per lane
  constexpr int kBlocks = kD / kRecurCols;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = blockIdx.x % kBlocks, h = (blockIdx.x / kBlocks) % a.Hv, s = blockIdx.x / (kBlocks * a.Hv);
  const int hk = h / (a.Hv / a.Hk);
  const int half = lane & 1, r0 = (lane >> 1) * kRows;
  const int col = blk * kRecurCols + warp * 8 + half * 4;
  // the total that this lane ends up with: of k (0) or q (1), of the pair's first or second token, for
  // column `mine` of its four; lanes of the u of that column
  const bool of_q = lane & 2, second = lane & 4;
  const int mine = (lane >> 3 & 1) * 2 + (lane >> 4 & 1);
  const int lane_u = lane & ~6;   // | 4: the second token's
  if (a.zero_rest) delta_zero_rest(a, a.out, a.Hv, kD);
  const DeltaSeq sq = delta_seq(a, s);
  // a token in shared memory: k, q, v of the block's columns, g, beta
  constexpr int kOffQ = kD * 2, kOffV = kD * 4, kOffG = kOffV + kRecurCols * 2, kToken = kOffG + 16;
  __shared__ __align__(16) uint8_t ring[2 * kRecurBatch * kToken];
  // what this thread copies of each batch: 16 bytes of a row (kIts of them at most), and one gate
  constexpr int kVec = kOffG / 16, kItems = kRecurBatch * kVec, kIts = (kItems + kRecurThreads - 1) / kRecurThreads;
  const int tid = threadIdx.x;
  const __nv_bfloat16* src[kIts];
  long long step[kIts];
  int token[kIts];
  uint32_t dst[kIts];
#pragma unroll
  for (int i = 0; i < kIts; ++i) {
    const int item = tid + i * kRecurThreads, t = item / kVec, c = item - t * kVec;
    const DeltaView& x = c < kOffQ / 16 ? a.k : c < kOffV / 16 ? a.q : a.v;
    const int at = c < kOffQ / 16 ? c * 8 : c < kOffV / 16 ? c * 8 - kD : blk * kRecurCols + c * 8 - 2 * kD;
    src[i] = delta_row(x, sq, t, c < kOffV / 16 ? hk : h) + at;
    step[i] = kRecurBatch * x.st;
    token[i] = item < kItems ? t : 1 << 30;   // (there are 2^30 tokens at most)
    dst[i] = smem_u32(ring + t * kToken + c * 16);
  }
  const int gate_token = tid < 2 * kRecurBatch ? tid >> 1 : 1 << 30;
  const long long gate_st = tid & 1 ? a.b_st : a.g_st;
  const float* gate = (tid & 1 ? a.beta + sq.entry * a.b_sb : a.g + sq.entry * a.g_sb) + (sq.first + (tid >> 1)) * gate_st + h;
  const uint32_t gate_dst = smem_u32(ring + (tid >> 1 & (kRecurBatch - 1)) * kToken + kOffG + (tid & 1) * 4);
  auto fetch = [&](int n0) {   // the next batch, tokens [n0, n0 + kRecurBatch), to its half of the ring
    const uint32_t o = n0 / kRecurBatch % 2 * (kRecurBatch * kToken);
#pragma unroll
    for (int i = 0; i < kIts; ++i) {
      if (n0 + token[i] < sq.len) cp_async_16(dst[i] + o, src[i], true);
      src[i] += step[i];
    }
    if (n0 + gate_token < sq.len) cp_async_4(gate_dst + o, gate);
    gate += kRecurBatch * gate_st;
    cp_async_commit();
  };
  fetch(0);
  const long long base = ((long long)s * a.Hv + h) * (long long)(kD * kD) + (long long)r0 * kD + col;
  F2 S[kRows][2];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.state_in != nullptr) x = *reinterpret_cast<const float4*>(a.state_in + base + (long long)j * kD);
    S[j][0] = f2(x.x, x.y), S[j][1] = f2(x.z, x.w);
  }
  __nv_bfloat16* op = const_cast<__nv_bfloat16*>(delta_row(a.out, sq, second, h)) + col + mine;
  for (int n = 0; n < sq.len; n += 2, op += 2 * a.out.st) {
    if (n % kRecurBatch == 0) {
      cp_async_wait<0>();
      __syncthreads();   // this batch is there, and all have left the one before it
      fetch(n + kRecurBatch);
    }
    const bool two = n + 1 < sq.len;   // else the second token is one that changes nothing
    const uint8_t* tok = ring + (n % (2 * kRecurBatch)) * kToken;
    float k[2][kRows], q[2][kRows], decay[2], write[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t kw[kRows / 2], qw[kRows / 2];
      const bool real = t == 0 || two;
      recur_load<kRows>(tok + t * kToken + r0 * 2, kw);
      recur_load<kRows>(tok + t * kToken + kOffQ + r0 * 2, qw);
      const float2 gates = *reinterpret_cast<const float2*>(tok + t * kToken + kOffG);
#pragma unroll
      for (int j = 0; j < kRows / 2; ++j) {
        if (!real) kw[j] = qw[j] = 0;
        k[t][2 * j] = __uint_as_float(kw[j] << 16), k[t][2 * j + 1] = __uint_as_float(kw[j] & 0xFFFF0000u);
        q[t][2 * j] = __uint_as_float(qw[j] << 16), q[t][2 * j + 1] = __uint_as_float(qw[j] & 0xFFFF0000u);
      }
      decay[t] = real ? expf(clamp_decay(gates.x)) : 1.f;
      write[t] = real ? gates.y : 0.f;
    }
    const bool has = !second || two;
    const float v = has ? bf16_up(reinterpret_cast<const uint16_t*>(tok + second * kToken + kOffV)[warp * 8 + half * 4 + mine]) : 0.f;
    // S^T k and S^T q of both tokens, of this lane's rows: [q][token][column]
    float sum[2][2][4];
    float dots[4] = {0.f, 0.f, 0.f, 0.f};   // k1 q1, k2 q2, k1 k2, k1 q2
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      F2 x[2] = {f2(0.f, 0.f), f2(0.f, 0.f)}, y[2] = {x[0], x[1]};
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const F2 k2 = f2(k[t][j], k[t][j]), q2 = f2(q[t][j], q[t][j]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          x[c] = f2_fma(S[j][c], k2, x[c]);
          y[c] = f2_fma(S[j][c], q2, y[c]);
        }
        dots[t] += k[t][j] * q[t][j];
        dots[2 + t] += k[0][j] * (t ? q[1][j] : k[1][j]);
      }
      const float2 x0 = f2_out(x[0]), x1 = f2_out(x[1]), y0 = f2_out(y[0]), y1 = f2_out(y[1]);
      sum[0][t][0] = x0.x, sum[0][t][1] = x0.y, sum[0][t][2] = x1.x, sum[0][t][3] = x1.y;
      sum[1][t][0] = y0.x, sum[1][t][1] = y0.y, sum[1][t][2] = y1.x, sum[1][t][3] = y1.y;
    }
    // each step halves what a lane holds: a lane keeps one half of its sums and gives the other one away
    auto halve = [&](bool up, float lo, float hi, int o) {
      return (up ? hi : lo) + __shfl_xor_sync(0xffffffffu, up ? lo : hi, o);
    };
    float total;
    {
      float x[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[t][c] = halve(of_q, sum[0][t][c], sum[1][t][c], 2);
#pragma unroll
      for (int c = 0; c < 4; ++c) x[0][c] = halve(second, x[0][c], x[1][c], 4);
      const float y0 = halve(mine & 2, x[0][0], x[0][2], 8), y1 = halve(mine & 2, x[0][1], x[0][3], 8);
      total = halve(mine & 1, y0, y1, 16);
    }
    {
      const float d0 = halve(lane & 2, dots[0], dots[1], 2), d1 = halve(lane & 2, dots[2], dots[3], 2);
      float d = halve(lane & 4, d0, d1, 4);
      d += __shfl_xor_sync(0xffffffffu, d, 8);
      d += __shfl_xor_sync(0xffffffffu, d, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) dots[i] = __shfl_sync(0xffffffffu, d, 2 * i);
    }
    const float both = decay[0] * decay[1], carried = (second ? both : decay[0]) * total;
    // u of the lane's token and column, where the total is k's
    float wrote = (second ? write[1] : write[0]) * (v - carried);
    const float first = __shfl_xor_sync(0xffffffffu, wrote, 4);
    if (second) wrote -= write[1] * decay[1] * dots[2] * first;
    F2 u[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = __shfl_sync(0xffffffffu, wrote, half | t << 2 | (c & 2) << 2 | (c & 1) << 4);
      u[t][0] = f2(x[0], x[1]), u[t][1] = f2(x[2], x[3]);
    }
    const float u1 = __shfl_sync(0xffffffffu, wrote, lane_u), u2 = __shfl_sync(0xffffffffu, wrote, lane_u | 4);
    if (of_q && has)
      *op = __float2bfloat16_rn(a.scale * (carried + (second ? decay[1] * dots[3] * u1 + dots[1] * u2 : dots[0] * u1)));
    const F2 d2 = f2(both, both);
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const float k1 = decay[1] * k[0][j];
      const F2 a2 = f2(k1, k1), b2 = f2(k[1][j], k[1][j]);
#pragma unroll
      for (int c = 0; c < 2; ++c) S[j][c] = f2_fma(b2, u[1][c], f2_fma(a2, u[0][c], f2_mul(d2, S[j][c])));
    }
  }
  if (a.state_out != nullptr)
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const float2 x = f2_out(S[j][0]), y = f2_out(S[j][1]);
      *reinterpret_cast<float4*>(a.state_out + base + (long long)j * kD) = make_float4(x.x, x.y, y.x, y.y);
    }
}

// ---------------------------------------------------------------------------------------
// litela_delta_step: one token, the serving form, on a pool of states: the recurrence's formulas.
//
// A state is read and written once, 8 d^2 bytes per head: HBM bound.  A CTA has 32 columns of a state,
// a warp a quarter of the rows, so that 8 lanes read 128 adjacent bytes; the warps' sums are added through
// shared memory.  96 rows of 32 heads of 128: 64 us, 6.4 TB/s (with the recurrence's layout, 32 bytes of
// 16 rows a load, the loads' wavefronts were at 67 % of their peak: 77 us); one row: 4.9 us.
template <int kD>
__global__ void __launch_bounds__(kRecurThreads, 6) litela_delta_step(const DeltaArgs a) {
  constexpr int kRows = kD / 16;   // rows per lane, 4 apart
  constexpr int kBlocks = kD / kRecurCols;
  constexpr int kWarps = kRecurThreads / 32;
  __shared__ __align__(16) float part[kWarps][2][kRecurCols];   // S^T k and S^T q of a warp's rows
  __shared__ float part_kq[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = blockIdx.x % kBlocks, h = (blockIdx.x / kBlocks) % a.Hv, s = blockIdx.x / (kBlocks * a.Hv);
  const int hk = h / (a.Hv / a.Hk);
  const int r0 = warp * (kD / kWarps) + (lane >> 3), c = (lane & 7) * 4, col = blk * kRecurCols + c;
  const DeltaSeq sq{s, 0, 1};
  const uint16_t* kp = reinterpret_cast<const uint16_t*>(delta_row(a.k, sq, 0, hk)) + r0;
  const uint16_t* qp = reinterpret_cast<const uint16_t*>(delta_row(a.q, sq, 0, hk)) + r0;
  float k[kRows], q[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) k[j] = bf16_up(kp[4 * j]), q[j] = bf16_up(qp[4 * j]);
  const uint2 vw = *reinterpret_cast<const uint2*>(delta_row(a.v, sq, 0, h) + col);
  const float decay = expf(clamp_decay(a.g[s * a.g_sb + h])), beta = a.beta[s * a.b_sb + h];
  long long slot = s;
  if (a.slots != nullptr) {
    // A row without a state of its own (an index outside the pool, or one that an earlier row has
    // already: its update would race with that row's) gets zeros and touches no state.
    slot = a.slots[s];
    bool dup = false;
    for (int i = threadIdx.x; i < s; i += kRecurThreads) dup |= a.slots[i] == (int)slot;
    if (__syncthreads_or(dup) || slot < 0 || slot >= a.nslots) {
      if (threadIdx.x < kRecurCols / 4)
        *reinterpret_cast<uint2*>(const_cast<__nv_bfloat16*>(delta_row(a.out, sq, 0, h)) + col) = make_uint2(0u, 0u);
      return;
    }
  }
  const long long base = (slot * a.Hv + h) * (long long)(kD * kD) + (long long)r0 * kD + col;
  F2 S[kRows][2];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.state_in != nullptr) x = *reinterpret_cast<const float4*>(a.state_in + base + (long long)j * 4 * kD);
    S[j][0] = f2(x.x, x.y), S[j][1] = f2(x.z, x.w);
  }
  F2 sk[2] = {f2(0.f, 0.f), f2(0.f, 0.f)}, sv[2] = {sk[0], sk[1]};
  float kq = 0.f;
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const F2 k2 = f2(k[j], k[j]), q2 = f2(q[j], q[j]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sk[i] = f2_fma(S[j][i], k2, sk[i]);
      sv[i] = f2_fma(S[j][i], q2, sv[i]);
    }
    kq += k[j] * q[j];
  }
  const float2 k01 = f2_out(sk[0]), k23 = f2_out(sk[1]), q01 = f2_out(sv[0]), q23 = f2_out(sv[1]);
  float x[4] = {k01.x, k01.y, k23.x, k23.y}, y[4] = {q01.x, q01.y, q23.x, q23.y};
  // lanes 0-7 and 16-23 go on with k's sums, the others with q's
  const bool of_q = lane & 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = (of_q ? y[i] : x[i]) + __shfl_xor_sync(0xffffffffu, of_q ? x[i] : y[i], 8);
    x[i] += __shfl_xor_sync(0xffffffffu, x[i], 16);
  }
  kq += __shfl_xor_sync(0xffffffffu, kq, 8);
  kq += __shfl_xor_sync(0xffffffffu, kq, 16);
  if (lane < 16) *reinterpret_cast<float4*>(&part[warp][of_q][c]) = make_float4(x[0], x[1], x[2], x[3]);
  if (lane == 0) part_kq[warp] = kq;
  __syncthreads();
  const float v[4] = {__uint_as_float(vw.x << 16), __uint_as_float(vw.x & 0xFFFF0000u), __uint_as_float(vw.y << 16),
                      __uint_as_float(vw.y & 0xFFFF0000u)};
  auto total = [&](int which, float* t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 p = *reinterpret_cast<const float4*>(&part[w][which][c]);
      t[0] += p.x, t[1] += p.y, t[2] += p.z, t[3] += p.w;
    }
  };
  float u[4], o[4];
  total(0, u);
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = beta * (v[i] - decay * u[i]);
  if (threadIdx.x < kRecurCols / 4) {
    total(1, o);
    const float all = part_kq[0] + part_kq[1] + part_kq[2] + part_kq[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = a.scale * (decay * o[i] + all * u[i]);
    __nv_bfloat162 lo = __floats2bfloat162_rn(o[0], o[1]), hi = __floats2bfloat162_rn(o[2], o[3]);
    *reinterpret_cast<uint2*>(const_cast<__nv_bfloat16*>(delta_row(a.out, sq, 0, h)) + col) =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  }
  if (a.state_out == nullptr) return;
  const F2 d2 = f2(decay, decay), u01 = f2(u[0], u[1]), u23 = f2(u[2], u[3]);
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const F2 k2 = f2(k[j], k[j]);
    const float2 l = f2_out(f2_fma(k2, u01, f2_mul(d2, S[j][0]))), r = f2_out(f2_fma(k2, u23, f2_mul(d2, S[j][1])));
    *reinterpret_cast<float4*>(a.state_out + base + (long long)j * 4 * kD) = make_float4(l.x, l.y, r.x, r.y);
  }
}

}  // namespace litela
