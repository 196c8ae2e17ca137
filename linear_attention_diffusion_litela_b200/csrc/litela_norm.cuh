// RMS norm of every query and key head and rotation by position, on packed q|k|v rows, and the
// gradient: one pass over the rows each.
//
// Per row (token) and head h of q or k, with x the head's d channels and w the weight of q or k:
//     r = 1 / sqrt(mean x^2 + eps),   y = R(pos) (w * r * x)
// R turns the first `rot` channels in pairs (a, b) by the position's angles:
//     (a, b) -> (a cos - b sin, b cos + a sin).
// Gradient, with t = R^T dy (the same pairs turned back):
//     dw = sum over rows and heads of t * r * x,   dx = r (w t - r x mean(w t * r x)).
// v passes through.
//
// Both are bound by HBM: a row is read once and written once, all sums are in fp32.  A lane owns
// 8 neighbouring channels (16 bytes); d / 8 lanes make a head and reduce with shuffles, so a warp
// takes 256 channels per step.  256 is a multiple of d, so a lane meets the same channels of a
// head in every step: its 8 cosines, sines and weights stay in registers for a whole row.  A warp
// takes a share of `parts` of a row; parts > 1 only where the rows alone do not fill the SMs.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "sm100_ptx.cuh"

namespace litela {

struct NormPlan {
  const __nv_bfloat16* x;      // [rows, W]
  const __nv_bfloat16* dy;     // backward
  __nv_bfloat16* out;          // y or dx, [rows, W]; may be x (forward) or dy (backward)
  const float* wq;             // [d] or null (ones)
  const float* wk;
  const float* cos;            // [table, rot / 2] or null (no rotation)
  const float* sin;
  const void* pos;             // [rows] int32 or int64, or null (the row's index in its batch entry)
  float* partials;             // backward: [grid][2][d] sums of the weights' gradients
  long long rows;
  int N;                       // tokens per batch entry
  int pos64, table, rot;
  int q_ch, qk_ch, W;          // first channel of k, of v, channels of a row
  int parts, steps;            // warps per row; 256-channel steps of a row
  bool copy_v;                 // out is another buffer than the input: v is copied
  float eps;
};

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kNormStep = 256;    // channels of a warp's step

__device__ __forceinline__ void bf16x8_to_f32(uint4 w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float* x) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// a row's position; a negative one marks a padded row
__device__ __forceinline__ long long norm_position(const NormPlan& p, long long row) {
  if (p.pos == nullptr) return row % p.N;
  return p.pos64 ? static_cast<const long long*>(p.pos)[row] : static_cast<const int*>(p.pos)[row];
}

// The lane's cosines and sines of channels [c, c + 8) of a head at position `at`.  Channels that
// are not rotated get (1, 0); a position behind the table gives NaN (the result shows it).
// Pairs: kInter, channels (2i, 2i + 1); else (i, i + rot / 2).  sn carries the sign of the
// partner's share, so that a channel's result is x * cs + partner * sn.
template <bool kInter>
__device__ __forceinline__ void norm_angles(const NormPlan& p, long long at, int c, float* cs, float* sn) {
  if (p.rot == 0 || c >= p.rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
    }
    return;
  }
  if (at >= p.table) {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __int_as_float(0x7fffffff);
    return;
  }
  const int half = p.rot / 2;
  if (kInter) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.cos + at * half + c / 2));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p.sin + at * half + c / 2));
    const float ca[4] = {a.x, a.y, a.z, a.w}, sa[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[2 * i] = cs[2 * i + 1] = ca[i];
      sn[2 * i] = -sa[i];
      sn[2 * i + 1] = sa[i];
    }
  } else {
    const bool second = c >= half;
    const long long o = at * half + (second ? c - half : c);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p.cos + o) + v);
      const float4 b = __ldg(reinterpret_cast<const float4*>(p.sin + o) + v);
      cs[4 * v] = a.x, cs[4 * v + 1] = a.y, cs[4 * v + 2] = a.z, cs[4 * v + 3] = a.w;
      sn[4 * v] = b.x, sn[4 * v + 1] = b.y, sn[4 * v + 2] = b.z, sn[4 * v + 3] = b.w;
    }
    if (!second)
#pragma unroll
      for (int i = 0; i < 8; ++i) sn[i] = -sn[i];
  }
}

// x * cs + partner * sn for the lane's 8 channels; `c` is the first of them in its head, `half`
// rot / 2 in lanes.  kBack turns back (the sines negated).  All lanes take part in the shuffles.
template <bool kInter, bool kBack, int kD>
__device__ __forceinline__ void norm_rotate(float* x, const float* cs, const float* sn, int rot, int lane) {
  if (rot == 0) return;
  float q[8];
  if (kInter) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = x[i ^ 1];
  } else {
    const int hl = rot / 16, l = lane % (kD / 8);   // lanes of half the rotated channels; lane in the head
    const int src = l < hl ? lane + hl : (l < 2 * hl ? lane - hl : lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __shfl_sync(0xffffffffu, x[i], src);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * cs[i] + (kBack ? -q[i] * sn[i] : q[i] * sn[i]);
}

__device__ __forceinline__ void load_weight(const float* w, int c, float* r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = w == nullptr ? 1.f : __ldg(w + c + i);
}

// this warp's part of a row of zeros
__device__ __forceinline__ void norm_zero_row(const NormPlan& p, __nv_bfloat16* dst, int part, int lane) {
  for (int s = part; s < p.steps; s += p.parts) {
    const int ch = s * kNormStep + lane * 8;
    if (ch < p.W) *reinterpret_cast<uint4*>(dst + ch) = make_uint4(0u, 0u, 0u, 0u);
  }
}

constexpr int kNormUnroll = 4;

template <int kD, bool kInter>
__global__ void __launch_bounds__(kNormThreads) litela_norm_fwd(const NormPlan p) {
  const int lane = threadIdx.x & 31;
  const long long nwarps = (long long)gridDim.x * kNormWarps;
  const int c = (lane * 8) % kD;
  float wq[8], wk[8];
  load_weight(p.wq, c, wq);
  load_weight(p.wk, c, wk);
  const int last = p.copy_v ? p.W : p.qk_ch;   // channels of a row that are written
  for (long long t = (long long)blockIdx.x * kNormWarps + (threadIdx.x >> 5); t < p.rows * p.parts; t += nwarps) {
    const long long row = t / p.parts;
    const int part = (int)(t - row * p.parts);
    const long long at = norm_position(p, row);
    const __nv_bfloat16* src = p.x + row * p.W;
    __nv_bfloat16* dst = p.out + row * p.W;
    if (at < 0) {   // a padded row
      if (p.copy_v) norm_zero_row(p, dst, part, lane);
      continue;
    }
    float cs[8], sn[8];
    norm_angles<kInter>(p, at, c, cs, sn);
    for (int s0 = part; s0 < p.steps; s0 += kNormUnroll * p.parts) {
      uint4 raw[kNormUnroll];
#pragma unroll
      for (int u = 0; u < kNormUnroll; ++u) {
        const int ch = (s0 + u * p.parts) * kNormStep + lane * 8;
        raw[u] = ch < last ? *reinterpret_cast<const uint4*>(src + ch) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < kNormUnroll; ++u) {
        const int first = (s0 + u * p.parts) * kNormStep, ch = first + lane * 8;
        if (first < p.qk_ch) {   // the same for the whole warp
          float x[8], ss = 0.f;
          bf16x8_to_f32(raw[u], x);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
          const float r = rsqrtf(sum_lanes<kD / 8>(ss) * (1.f / kD) + p.eps);
          const bool q = ch < p.q_ch;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= r * (q ? wq[i] : wk[i]);
          norm_rotate<kInter, false, kD>(x, cs, sn, p.rot, lane);
          if (ch < p.qk_ch) raw[u] = f32_to_bf16x8(x);
        }
        if (ch < last) *reinterpret_cast<uint4*>(dst + ch) = raw[u];
      }
    }
  }
}

// The gradient.  A warp's sums of the weights' gradients stay in registers over all its rows; the
// CTA's sums go to `partials`, which litela_norm_weight_grad adds in a fixed order.
template <int kD, bool kInter>
__global__ void __launch_bounds__(kNormThreads) litela_norm_bwd(const NormPlan p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long nwarps = (long long)gridDim.x * kNormWarps;
  const int c = (lane * 8) % kD;
  float wq[8], wk[8], aq[8], ak[8];
  load_weight(p.wq, c, wq);
  load_weight(p.wk, c, wk);
#pragma unroll
  for (int i = 0; i < 8; ++i) aq[i] = ak[i] = 0.f;
  const int last = p.copy_v ? p.W : p.qk_ch;
  for (long long t = (long long)blockIdx.x * kNormWarps + warp; t < p.rows * p.parts; t += nwarps) {
    const long long row = t / p.parts;
    const int part = (int)(t - row * p.parts);
    const long long at = norm_position(p, row);
    __nv_bfloat16* dst = p.out + row * p.W;
    if (at < 0) {   // a padded row: its gradient is zero
      norm_zero_row(p, dst, part, lane);
      continue;
    }
    float cs[8], sn[8];
    norm_angles<kInter>(p, at, c, cs, sn);
    const __nv_bfloat16 *src = p.x + row * p.W, *grad = p.dy + row * p.W;
    constexpr int kU = kNormUnroll / 2;
    for (int s0 = part; s0 < p.steps; s0 += kU * p.parts) {
      uint4 rx[kU], rg[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int ch = (s0 + u * p.parts) * kNormStep + lane * 8;
        rx[u] = ch < p.qk_ch ? *reinterpret_cast<const uint4*>(src + ch) : make_uint4(0u, 0u, 0u, 0u);
        rg[u] = ch < last ? *reinterpret_cast<const uint4*>(grad + ch) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int first = (s0 + u * p.parts) * kNormStep, ch = first + lane * 8;
        if (first < p.qk_ch) {
          float x[8], g[8], ss = 0.f, dot = 0.f;
          bf16x8_to_f32(rx[u], x);
          bf16x8_to_f32(rg[u], g);
          norm_rotate<kInter, true, kD>(g, cs, sn, p.rot, lane);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
          const float r = rsqrtf(sum_lanes<kD / 8>(ss) * (1.f / kD) + p.eps);
          const bool q = ch < p.q_ch;
          const bool real = ch < p.qk_ch;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] *= r;
            const float gw = real ? g[i] * x[i] : 0.f;
            aq[i] += q ? gw : 0.f;
            ak[i] += q ? 0.f : gw;
            g[i] *= q ? wq[i] : wk[i];
            dot += g[i] * x[i];
          }
          dot = sum_lanes<kD / 8>(dot) * (1.f / kD);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = r * (g[i] - x[i] * dot);
          if (real) rg[u] = f32_to_bf16x8(x);
        }
        if (ch < last) *reinterpret_cast<uint4*>(dst + ch) = rg[u];
      }
    }
  }
  if (p.partials == nullptr) return;
  // lanes of the same channels, then the CTA's warps
  __shared__ float sums[kNormWarps][2][kD];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int o = kD / 8; o < 32; o <<= 1) {
      aq[i] += __shfl_xor_sync(0xffffffffu, aq[i], o);
      ak[i] += __shfl_xor_sync(0xffffffffu, ak[i], o);
    }
    if (lane < kD / 8) {
      sums[warp][0][lane * 8 + i] = aq[i];
      sums[warp][1][lane * 8 + i] = ak[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kD; i += kNormThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kNormWarps; ++w) s += sums[w][i / kD][i % kD];
    p.partials[(long long)blockIdx.x * 2 * kD + i] = s;
  }
}

// dw[i] = sum over the CTAs' partial sums, in a fixed order: one warp per element
__global__ void __launch_bounds__(32) litela_norm_weight_grad(const float* __restrict__ partials, int count, int d,
                                                             float* dwq, float* dwk) {
  sm100::pdl_wait_primary();
  const int i = blockIdx.x;
  float s = 0.f;
  for (int k = threadIdx.x; k < count; k += 32) s += __ldcg(partials + (long long)k * 2 * d + i);
  s = sum_lanes<32>(s);
  float* dw = i < d ? dwq : dwk;
  if (threadIdx.x == 0 && dw != nullptr) dw[i % d] = s;
}

}  // namespace litela
