// The gated delta rule: arguments shared by its kernels, and the recurrent kernel.
//
// Per sequence and value head (key head = value head / group), with q, k the key head's d
// channels, v the value head's, g the log decay and beta the write strength of a token, and a
// d x d state S (rows: key channels, columns: value channels):
//     S <- e^g S + k (beta (v - e^g S^T k))^T,     out = scale * S^T q.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

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

// ---------------------------------------------------------------------------------------
// litela_delta_recur: the recurrence, one token after another, the state in registers.
//
// A warp owns 8 columns of one state (all d rows): lane = row group (lane / 2) and 4 columns
// (lane & 1), rows lane / 2 + 16 j.  Nothing is shared between warps.  S^T k and S^T q of the
// state before the token are summed in the same shuffles: with them
//     u = beta (v - e^g S^T k),   out = scale * (e^g S^T q + (k . q) u),   S <- e^g S + k u^T,
// so that the update of S is off the way from one token's sums to the next one's output.
// One token (the serving form) moves a state once in and once out, 8 d^2 bytes per head: HBM
// bound.  The grid is one CTA per 32 columns, so that one sequence already fills the SMs.
// More tokens: bound by the ~0.3 us between one token's loads and the next one's.
constexpr int kRecurThreads = 128;
constexpr int kRecurCols = 32;

template <int kD>
__global__ void __launch_bounds__(kRecurThreads) litela_delta_recur(const DeltaArgs a) {
  constexpr int kRows = kD / 16;   // rows per lane
  constexpr int kBlocks = kD / kRecurCols;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = blockIdx.x % kBlocks, h = (blockIdx.x / kBlocks) % a.Hv, s = blockIdx.x / (kBlocks * a.Hv);
  const int hk = h / (a.Hv / a.Hk);
  const int col = blk * kRecurCols + warp * 8 + (lane & 1) * 4, r0 = lane >> 1;
  const DeltaSeq sq = delta_seq(a, s);
  long long slot = s;
  if (a.slots != nullptr) {
    // A row without a state of its own (an index outside the pool, or one that an earlier row has
    // already: its update would race with that row's) gets zeros and touches no state.
    slot = a.slots[s];
    bool dup = false;
    for (int i = threadIdx.x; i < s; i += kRecurThreads) dup |= a.slots[i] == (int)slot;
    if (__syncthreads_or(dup) || slot < 0 || slot >= a.nslots) {
      for (int n = 0; n < sq.len; ++n)
        if (threadIdx.x < kRecurCols / 4) {
          __nv_bfloat16* o = const_cast<__nv_bfloat16*>(delta_row(a.out, sq, n, h)) + blk * kRecurCols + threadIdx.x * 4;
          *reinterpret_cast<uint2*>(o) = make_uint2(0u, 0u);
        }
      return;
    }
  }
  const long long base = (slot * a.Hv + h) * (long long)(kD * kD) + (long long)r0 * kD + col;
  float S[kRows][4];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.state_in != nullptr) x = *reinterpret_cast<const float4*>(a.state_in + base + (long long)j * 16 * kD);
    S[j][0] = x.x, S[j][1] = x.y, S[j][2] = x.z, S[j][3] = x.w;
  }
  for (int n = 0; n < sq.len; ++n) {
    const uint16_t* kp = reinterpret_cast<const uint16_t*>(delta_row(a.k, sq, n, hk)) + r0;
    const uint16_t* qp = reinterpret_cast<const uint16_t*>(delta_row(a.q, sq, n, hk)) + r0;
    const long long tok = sq.first + n;
    const float decay = expf(clamp_decay(a.g[sq.entry * a.g_sb + tok * a.g_st + h]));
    const float beta = a.beta[sq.entry * a.b_sb + tok * a.b_st + h];
    const uint2 vr = *reinterpret_cast<const uint2*>(delta_row(a.v, sq, n, h) + col);
    float k[kRows], q[kRows], sum[9];
#pragma unroll
    for (int i = 0; i < 9; ++i) sum[i] = 0.f;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      k[j] = bf16_up(kp[16 * j]);
      q[j] = bf16_up(qp[16 * j]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        sum[c] += S[j][c] * k[j];
        sum[4 + c] += S[j][c] * q[j];
      }
      sum[8] += k[j] * q[j];
    }
#pragma unroll
    for (int i = 0; i < 9; ++i)
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    const float v[4] = {__uint_as_float(vr.x << 16), __uint_as_float(vr.x & 0xFFFF0000u),
                        __uint_as_float(vr.y << 16), __uint_as_float(vr.y & 0xFFFF0000u)};
    float u[4], o[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u[c] = beta * (v[c] - decay * sum[c]);
      o[c] = a.scale * (decay * sum[4 + c] + sum[8] * u[c]);
    }
    if (r0 == 0) {
      __nv_bfloat162 lo = __floats2bfloat162_rn(o[0], o[1]), hi = __floats2bfloat162_rn(o[2], o[3]);
      *reinterpret_cast<uint2*>(const_cast<__nv_bfloat16*>(delta_row(a.out, sq, n, h)) + col) =
          make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[j][c] = decay * S[j][c] + k[j] * u[c];
  }
  if (a.state_out != nullptr)
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      *reinterpret_cast<float4*>(a.state_out + base + (long long)j * 16 * kD) =
          make_float4(S[j][0], S[j][1], S[j][2], S[j][3]);
}

// zeros in the rows of a packed [token, head, d] output that no sequence has: those before the
// first one and behind the last one
__global__ void __launch_bounds__(256) litela_delta_zero_tail(const DeltaView out, const int* cu, int nseq, int ntok,
                                                             int heads, int d) {
  const int b = min(max(cu[0], 0), ntok), e = min(max(cu[nseq], b), ntok);
  const int per_row = heads * (d / 8);
  const long long n = (long long)(b + ntok - e) * per_row;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const int row = (int)(i / per_row), c = (int)(i - (long long)row * per_row);
    const int t = row < b ? row : e + row - b;
    *reinterpret_cast<uint4*>(out.p + (long long)t * out.st + (c / (d / 8)) * out.sh + (c % (d / 8)) * 8) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

}  // namespace litela
