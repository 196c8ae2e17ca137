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
// head in every step.  Work is cut by row and by q, k and v, all rows' q first: within a task the
// weight and the angles of a lane's channels are constants in registers, and the weight's gradient
// is one set of 8 sums.  Loads of a warp's next steps (of its next task, too) are in flight while
// it works on the ones before.  `parts` warps share a task; more than one only where the tasks alone
// do not fill the SMs.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "f32x2.cuh"
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
  int shift;                   // 2^shift warps share a task
  int regions;                 // 2: q and k; 3: v too
  bool copy_v;                 // out is another buffer than the input: v is copied
  float eps;
};

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kNormStep = 256;    // channels of a warp's step
constexpr int kNormAhead = 5120;  // bytes of a task that is fetched ahead, at most (norm_prefetch)

template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A row's position; a negative one marks a padded row.  Loaded as its words first, so that nothing
// waits for it before it is used.
__device__ __forceinline__ int2 norm_position_words(const NormPlan& p, long long row) {
  if (p.pos == nullptr)
    return make_int2((int)(p.rows <= 0xffffffffLL ? (uint32_t)row % (uint32_t)p.N : row % p.N), 0);
  if (p.pos64) return static_cast<const int2*>(p.pos)[row];
  return make_int2(static_cast<const int*>(p.pos)[row], 0);
}
__device__ __forceinline__ long long norm_position(const NormPlan& p, int2 w) {
  return p.pos64 ? (long long)((uint64_t)(uint32_t)w.y << 32 | (uint32_t)w.x) : w.x;
}

// Where a warp is: task t (region 0, 1, 2 = q, k, v of a row that starts at element `row` and has
// position `at`), channels [ch, end) of it to go
struct NormWalk {
  long long t, row;
  int2 at;
  int region, ch, end;
};

__device__ __forceinline__ void norm_task(const NormPlan& p, NormWalk& w) {
  const long long each = p.rows << p.shift;
  long long i = w.t;
  w.region = 0;
  if (i >= each) i -= each, w.region = 1;
  if (i >= each) i -= each, w.region = 2;
  w.at = norm_position_words(p, i >> p.shift);
  w.row = (i >> p.shift) * p.W;
  w.ch = (w.region == 0 ? 0 : w.region == 1 ? p.q_ch : p.qk_ch) + (int)(i & ((1 << p.shift) - 1)) * kNormStep;
  w.end = w.region == 0 ? p.q_ch : w.region == 1 ? p.qk_ch : p.W;
}

// to the next channels of a task, kU steps on, or to the next task that has any; false behind the last
template <int kU>
__device__ __forceinline__ bool norm_next(const NormPlan& p, NormWalk& w, long long nwarps) {
  w.ch += (kU * kNormStep) << p.shift;
  while (w.ch >= w.end) {
    w.t += nwarps;
    if (w.t >= (p.rows << p.shift) * p.regions) return false;
    norm_task(p, w);
  }
  return true;
}

// A whole task's channels into L2, one task ahead of the forward's loads: more bytes in flight than
// registers hold.  Tasks of 2240 and 4480 bytes: 206 -> 174 us, 184 -> 164 us (60000 rows of 3 x 35, 32768 of
// 3 x 70 heads of 32); of 8192 and 16384 bytes, whose own loads are enough: 244 -> 322 us, 268 -> 377 us, and the
// gradient (two rows a task) 62 -> 70 us: not fetched.  Nothing between 4480 and 8192 bytes was measured.
__device__ __forceinline__ void norm_prefetch(const NormPlan& p, long long t, int lane) {
  if (p.shift != 0 || lane != 0 || t >= p.rows * p.regions) return;
  const int region = (t >= p.rows) + (t >= 2 * p.rows);
  const int first = region == 0 ? 0 : region == 1 ? p.q_ch : p.qk_ch;
  const int bytes = ((region == 0 ? p.q_ch : region == 1 ? p.qk_ch : p.W) - first) * 2;
  if (bytes > 0 && bytes <= kNormAhead) sm100::bulk_prefetch_l2(p.x + (t - region * p.rows) * p.W + first, bytes);
}

template <int kU>
__device__ __forceinline__ void norm_load(const NormPlan& p, const __nv_bfloat16* x, const NormWalk& w, int lane,
                                          uint4* raw) {
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int ch = w.ch + ((u * kNormStep) << p.shift) + lane * 8;
    raw[u] = ch < w.end ? *reinterpret_cast<const uint4*>(x + w.row + ch) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// The lane's cosines and sines of channels [c, c + 8) of a head at position `at`.  Channels that
// are not rotated get (1, 0); a position behind the table gives NaN (the result shows it).
// Pairs: kInter, channels (2i, 2i + 1); else (i, i + rot / 2).  sn carries the sign of the
// partner's share, so that a channel's result is x * cs + partner * sn.
template <bool kInter>
__device__ __forceinline__ void norm_angles(const NormPlan& p, long long at, int c, F2* cs, F2* sn) {
  if (c >= p.rot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = f2(1.f, 1.f), sn[i] = f2(0.f, 0.f);
    return;
  }
  if (at >= p.table) {
    const float nan = __int_as_float(0x7fffffff);
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = sn[i] = f2(nan, nan);
    return;
  }
  const int half = p.rot / 2;
  if (kInter) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.cos + at * half + c / 2));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p.sin + at * half + c / 2));
    cs[0] = f2(a.x, a.x), cs[1] = f2(a.y, a.y), cs[2] = f2(a.z, a.z), cs[3] = f2(a.w, a.w);
    sn[0] = f2(-b.x, b.x), sn[1] = f2(-b.y, b.y), sn[2] = f2(-b.z, b.z), sn[3] = f2(-b.w, b.w);
  } else {
    const bool second = c >= half;
    const long long o = at * half + (second ? c - half : c);
    const F2 sign = second ? f2(1.f, 1.f) : f2(-1.f, -1.f);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p.cos + o) + v);
      const float4 b = __ldg(reinterpret_cast<const float4*>(p.sin + o) + v);
      cs[2 * v] = f2(a.x, a.y), cs[2 * v + 1] = f2(a.z, a.w);
      sn[2 * v] = f2_mul(sign, f2(b.x, b.y)), sn[2 * v + 1] = f2_mul(sign, f2(b.z, b.w));
    }
  }
}

// 8 bf16 values of the lane's channels' partners; all lanes take part.  src: norm_partner
template <bool kInter>
__device__ __forceinline__ uint4 norm_swap(uint4 w, int src) {
  if (kInter) {
    auto turn = [](uint32_t v) { return __funnelshift_l(v, v, 16); };
    return make_uint4(turn(w.x), turn(w.y), turn(w.z), turn(w.w));
  }
  return make_uint4(__shfl_sync(0xffffffffu, w.x, src), __shfl_sync(0xffffffffu, w.y, src),
                    __shfl_sync(0xffffffffu, w.z, src), __shfl_sync(0xffffffffu, w.w, src));
}
// the lane that holds the partners (pairs of two halves), itself for channels that are not rotated
template <int kD>
__device__ __forceinline__ int norm_partner(int rot, int lane) {
  const int hl = rot / 16, l = lane % (kD / 8);   // lanes of half the rotated channels; lane in the head
  return l < hl ? lane + hl : l < 2 * hl ? lane - hl : lane;
}

__device__ __forceinline__ void f2_bf16x8(uint4 w, F2* x) {
  x[0] = f2_bf16(w.x), x[1] = f2_bf16(w.y), x[2] = f2_bf16(w.z), x[3] = f2_bf16(w.w);
}
__device__ __forceinline__ uint4 f2_to_bf16x8(const F2* x) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = f2_out(x[i]);
    __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    u[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ float f2_sum4(const F2* x) {
  const float2 v = f2_out(f2_add(f2_add(x[0], x[1]), f2_add(x[2], x[3])));
  return v.x + v.y;
}

// both weights, ones where there are none
template <int kD>
__device__ __forceinline__ void norm_weights(const NormPlan& p, float (*w)[kD]) {
  for (int i = threadIdx.x; i < 2 * kD; i += kNormThreads) {
    const float* src = i < kD ? p.wq : p.wk;
    w[i / kD][i % kD] = src == nullptr ? 1.f : __ldg(src + i % kD);
  }
  __syncthreads();
}

// this warp's steps of the walk's channels, zeros
template <int kU>
__device__ __forceinline__ void norm_zero(const NormPlan& p, const NormWalk& w, int lane) {
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int ch = w.ch + ((u * kNormStep) << p.shift) + lane * 8;
    if (ch < w.end) *reinterpret_cast<uint4*>(p.out + w.row + ch) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// y = r (x * a + partner * b), a = w cos, b = the partner's w times the signed sine.  80 registers
// (three CTAs an SM) hold four steps in work and four in flight.  2 x 16384 rows of 70 + 70 + 70
// heads of 32 channels: 158 us, 5.6 TB/s (176 without norm_prefetch, 179 with 64 registers, two steps and
// four CTAs); neither the issue slots (59 %) nor DRAM (67 %) are full, warps wait for loads most.
template <int kD, bool kInter>
__global__ void __launch_bounds__(kNormThreads, 3) litela_norm_fwd(const NormPlan p) {
  constexpr int kU = 4;
  __shared__ float weight[2][kD];
  const int lane = threadIdx.x & 31;
  const long long nwarps = (long long)gridDim.x * kNormWarps;
  const int c = (lane * 8) % kD, src = norm_partner<kD>(p.rot, lane);
  NormWalk to{(long long)blockIdx.x * kNormWarps + (threadIdx.x >> 5) - nwarps, 0, {}, 0, 0, 0};
  bool more = norm_next<kU>(p, to, nwarps);
  uint4 ahead[kU];
  if (more) norm_load<kU>(p, p.x, to, lane, ahead);
  norm_weights<kD>(p, weight);
  long long task = -1, pos = 0;
  F2 a[4], b[4];
  while (more) {
    const NormWalk w = to;
    uint4 raw[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) raw[u] = ahead[u];
    more = norm_next<kU>(p, to, nwarps);
    if (more) norm_load<kU>(p, p.x, to, lane, ahead);
    if (w.t != task) {
      task = w.t;
      norm_prefetch(p, task + nwarps, lane);
      pos = norm_position(p, w.at);
      if (pos >= 0 && w.region < 2) {
        norm_angles<kInter>(p, pos, c, a, b);
        const float* wt = weight[w.region];
        const int pc = kInter ? c : c + (src - lane) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 own = *reinterpret_cast<const float2*>(wt + c + 2 * i);
          const float2 oth = *reinterpret_cast<const float2*>(wt + pc + 2 * i);
          a[i] = f2_mul(a[i], f2(own.x, own.y));
          b[i] = f2_mul(b[i], kInter ? f2(oth.y, oth.x) : f2(oth.x, oth.y));
        }
      }
    }
    if (pos < 0) {   // a padded row
      if (p.copy_v) norm_zero<kU>(p, w, lane);
      continue;
    }
    auto step = [&](int u, bool heads) {
      const int ch = w.ch + ((u * kNormStep) << p.shift) + lane * 8;
      if (heads) {
        F2 x[4], q[4], s[4];
        f2_bf16x8(raw[u], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = f2_mul(x[i], x[i]);
        const float r = rsqrtf(sum_lanes<kD / 8>(f2_sum4(s)) * (1.f / kD) + p.eps);
        const F2 r2 = f2(r, r);
        if (p.rot != 0) {
          f2_bf16x8(norm_swap<kInter>(raw[u], src), q);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = f2_fma(x[i], a[i], f2_mul(q[i], b[i]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = f2_mul(x[i], a[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2_mul(r2, x[i]);
        raw[u] = f2_to_bf16x8(x);
      }
      if (ch < w.end) *reinterpret_cast<uint4*>(p.out + w.row + ch) = raw[u];
    };
    if (w.region == 2) {
#pragma unroll
      for (int u = 0; u < kU; ++u) step(u, false);
    } else if (w.ch + (((kU - 1) * kNormStep) << p.shift) < w.end) {   // all steps are there: they interleave
#pragma unroll
      for (int u = 0; u < kU; ++u) step(u, true);
    } else {
#pragma unroll
      for (int u = 0; u < kU - 1; ++u) {
        if (w.ch + ((u * kNormStep) << p.shift) >= w.end) break;
        step(u, true);
      }
    }
  }
}

// The gradient.  With t the turned-back dy: dw = sum of r t x, dx = r (w t - x r^2 mean(w t x)), so
// that the two sums of a head do not wait for one another.  A warp's sums of a weight's gradient
// stay in registers over all its rows; the CTA's go to `partials`, which litela_norm_weight_grad
// adds in a fixed order.  Two CTAs an SM with two steps in work and two in flight: 2 x 4099 rows of
// 32 + 8 + 8 heads of 128 channels in 62 us, 4.7 TB/s (80 registers for a third CTA spill: 144 us).  With 15.5 warps an
// SM too few bytes are in flight: 58 % of the issue slots, 49 % of DRAM.
template <int kD, bool kInter>
__global__ void __launch_bounds__(kNormThreads, 2) litela_norm_bwd(const NormPlan p) {
  constexpr int kU = 2;
  __shared__ float weight[2][kD];
  __shared__ float sums[kNormWarps][2][kD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long nwarps = (long long)gridDim.x * kNormWarps;
  const int c = (lane * 8) % kD, src = norm_partner<kD>(p.rot, lane);
  NormWalk to{(long long)blockIdx.x * kNormWarps + warp - nwarps, 0, {}, 0, 0, 0};
  uint4 ax[kU], ag[kU];
  auto load = [&] {
    if (to.region < 2) norm_load<kU>(p, p.x, to, lane, ax);
    if (to.region < 2 || p.copy_v) norm_load<kU>(p, p.dy, to, lane, ag);
  };
  bool more = norm_next<kU>(p, to, nwarps);
  if (more) load();
  norm_weights<kD>(p, weight);
  for (int i = threadIdx.x; i < kNormWarps * 2 * kD; i += kNormThreads) (&sums[0][0][0])[i] = 0.f;
  __syncthreads();
  F2 acc[4], cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = f2(0.f, 0.f);
  // the sums of region r so far: lanes of the same channels added, and left to the CTA
  auto put = [&](int r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 v = f2_out(acc[i]);
#pragma unroll
      for (int o = kD / 8; o < 32; o <<= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      }
      if (lane < kD / 8) sums[warp][r][c + 2 * i] = v.x, sums[warp][r][c + 2 * i + 1] = v.y;
      acc[i] = f2(0.f, 0.f);
    }
  };
  long long task = -1, pos = 0;
  int region = 0;
  while (more) {
    const NormWalk w = to;
    uint4 rx[kU], rg[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) rx[u] = ax[u], rg[u] = ag[u];
    more = norm_next<kU>(p, to, nwarps);
    if (more) load();
    if (w.t != task) {
      task = w.t;
      pos = norm_position(p, w.at);
      if (w.region != region) {
        if (region < 2) put(region);
        region = w.region;
      }
      if (pos >= 0 && w.region < 2) {
        norm_angles<kInter>(p, pos, c, cs, sn);
#pragma unroll
        for (int i = 0; i < 4; ++i) sn[i] = f2_mul(f2(-1.f, -1.f), sn[i]);   // back
      }
    }
    if (pos < 0) {   // a padded row: its gradient is zero
      norm_zero<kU>(p, w, lane);
      continue;
    }
    if (w.region == 2 && !p.copy_v) continue;
    auto step = [&](int u, bool heads) {
      const int ch = w.ch + ((u * kNormStep) << p.shift) + lane * 8;
      if (heads) {
        F2 x[4], g[4], s[4], d[4], e[4];
        f2_bf16x8(rx[u], x);
        f2_bf16x8(rg[u], g);
        if (p.rot != 0) {
          F2 q[4];
          f2_bf16x8(norm_swap<kInter>(rg[u], src), q);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = f2_fma(g[i], cs[i], f2_mul(q[i], sn[i]));
        }
        const float* wt = weight[w.region] + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 wv = *reinterpret_cast<const float2*>(wt + 2 * i);
          s[i] = f2_mul(x[i], x[i]);
          d[i] = f2_mul(g[i], x[i]);
          g[i] = f2_mul(g[i], f2(wv.x, wv.y));
          e[i] = f2_mul(g[i], x[i]);
        }
        const float ss = sum_lanes<kD / 8>(f2_sum4(s)), dot = sum_lanes<kD / 8>(f2_sum4(e));
        const float r = rsqrtf(ss * (1.f / kD) + p.eps), m = -(dot * (1.f / kD) * r);
        const F2 r2 = f2(r, r), m2 = f2(m, m);
        if (ch < w.end)   // r may be infinite behind the last head
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = f2_fma(d[i], r2, acc[i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2_mul(r2, f2_fma(f2_mul(x[i], r2), m2, g[i]));
        rg[u] = f2_to_bf16x8(x);
      }
      if (ch < w.end) *reinterpret_cast<uint4*>(p.out + w.row + ch) = rg[u];
    };
    if (w.region == 2) {
#pragma unroll
      for (int u = 0; u < kU; ++u) step(u, false);
    } else if (w.ch + (((kU - 1) * kNormStep) << p.shift) < w.end) {   // all steps are there: they interleave
#pragma unroll
      for (int u = 0; u < kU; ++u) step(u, true);
    } else {
#pragma unroll
      for (int u = 0; u < kU - 1; ++u) {
        if (w.ch + ((u * kNormStep) << p.shift) >= w.end) break;
        step(u, true);
      }
    }
  }
  if (p.partials == nullptr) return;
  if (region < 2) put(region);
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
