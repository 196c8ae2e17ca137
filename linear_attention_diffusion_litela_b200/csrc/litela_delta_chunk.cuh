// The gated delta rule over whole sequences, in chunks of 64 tokens.
//
// With G_i the sum of the log decays of a chunk's tokens up to i, S0 the state before the chunk,
// D_ij = e^(G_i - G_j) for i >= j, and the chunk's rows as matrices K, Q, V [64, d]:
//     A = diag(beta) (K K^T . D) below the diagonal,  T = (I + A)^-1,  P = scale (Q K^T . D)
//     R = diag(beta) (V - diag(e^G) K S0),            U = T R            (the written values)
//     out = scale diag(e^G) Q S0 + P T R,             S = e^G_C S0 + K^T diag(e^(G_C - G)) U.
// T and P T need no state: litela_delta_prep makes them for all chunks at once.  What is left of
// a chunk are three products that follow one another, and litela_delta_chain walks a sequence's
// chunks with them.
//
// Precision.  States are fp32 and stay in registers.  An fp32 operand of a tensor-core product is
// entered as a bf16 pair (hi + lo, 2^-17 relative) and the products hi*hi, hi*lo, lo*hi are summed
// in fp32: a single bf16 rounding (2^-8) of T, R, U or S0 would show in the states.  K, Q and V are
// bf16 already.  G is summed in fp64: differences of large sums of decays would lose in fp32.
//
// A NaN or an infinity must not reach the tokens before its own: 0 * NaN inside a product would
// carry it there.  So non-finite entries are taken out of A, P and R, the first token that had one
// is kept, and it and all later tokens of the sequence (and the state) get NaN.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "litela_delta.cuh"
#include "sm100_ptx.cuh"

namespace litela {

constexpr int kChunk = 64;

// One chunk and value head's prepared block: [T; P T] as the A operand image of a tcgen05 product
// (128 rows x 64 columns bf16, K-major, 128-byte swizzle), hi then lo, then per-token factors
constexpr uint32_t kImgHalf = 128 * 128;
constexpr uint32_t kPrepFactors = 2 * kImgHalf;
constexpr uint32_t kPrepBytes = kPrepFactors + 1024;
// fp32 at kPrepFactors: e^G [64], e^(G_C - G) [64] (0 behind the end), beta [64] (0 behind the
// end), then e^G_C and (int32) the first token of the chunk with a non-finite A or P, or 64
constexpr int kFacDecay = 0, kFacToEnd = 64, kFacBeta = 128, kFacChunk = 192, kFacBad = 193;

// Chunk slots.  A batch of equal lengths: sequence s has the slots s * ceil(N / 64) + c.  Packed:
// cu[s] / 64 + s + c, which leaves every sequence at least ceil(len / 64) slots without a sum
// over the lengths before it; N / 64 + sequences slots in all, some of them empty.
__host__ __device__ inline long long delta_slots(int nseq, int ntok, bool packed) {
  return packed ? (long long)ntok / kChunk + nseq : (long long)nseq * ((ntok + kChunk - 1) / kChunk);
}
__device__ __forceinline__ long long delta_slot0(const DeltaArgs& a, int s, const DeltaSeq& q) {
  return a.cu == nullptr ? (long long)s * ((a.ntok + kChunk - 1) / kChunk) : (long long)q.first / kChunk + s;
}

// The sequence of a slot and its chunk there (whole warp); false for an empty slot.
__device__ __forceinline__ bool delta_find(const DeltaArgs& a, long long slot, int lane, int& s, DeltaSeq& q, int& n0) {
  if (a.cu == nullptr) {
    const int nc = (a.ntok + kChunk - 1) / kChunk;
    s = (int)(slot / nc);
    q = delta_seq(a, s);
    n0 = (int)(slot - (long long)s * nc) * kChunk;
    return true;
  }
  int lo = 0, hi = a.nseq;   // the last s with cu[s] / 64 + s <= slot is in [lo, hi)
  while (true) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool below = at < hi && (long long)(min(max(a.cu[at], 0), a.ntok) / kChunk) + at <= slot;
    const int n = __popc(__ballot_sync(0xffffffffu, below));
    if (n == 0) return false;
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) break;
  }
  s = lo;
  q = delta_seq(a, s);
  n0 = (int)(slot - delta_slot0(a, s, q)) * kChunk;
  return n0 >= 0 && n0 < q.len;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
// (a, b) as bf16 pairs: hi, and what hi leaves
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(a, b);
  lo = pack_bf16(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
}
// 16 x 16 accumulators (two 16 x 8 tiles) as an A operand, hi and lo
__device__ __forceinline__ void split_frag(const float (*c)[4], uint32_t* hi, uint32_t* lo) {
  split_bf16(c[0][0], c[0][1], hi[0], lo[0]);
  split_bf16(c[0][2], c[0][3], hi[1], lo[1]);
  split_bf16(c[1][0], c[1][1], hi[2], lo[2]);
  split_bf16(c[1][2], c[1][3], hi[3], lo[3]);
}
// D += A B with both as bf16 pairs
__device__ __forceinline__ void mma_split(float* d, const uint32_t* ahi, const uint32_t* alo, const uint32_t* bhi,
                                          const uint32_t* blo) {
  sm100::mma_16816(d, ahi, bhi);
  sm100::mma_16816(d, ahi, blo);
  sm100::mma_16816(d, alo, bhi);
}

// byte offset of bf16 element (row, column < 64) in a tile of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t sw128(int row, int col) {
  return (uint32_t)(row * 128 + ((((col >> 3) ^ row) & 7) << 4) + (col & 7) * 2);
}

// ---------------------------------------------------------------------------------------
// litela_delta_prep: T and P T of one chunk and value head per CTA, 4 warps, warp w the rows
// 16 w .. 16 w + 15.
//
// mma.sync: the operands are one chunk's, 64 rows, and T is made of 16 x 16 blocks where each
// product waits for the one before; a tcgen05 product would be a sixth full and go through TMEM and
// shared memory for each block.  T by blocks of 16: the diagonal blocks by substitution, one lane
// a column; below them, block column j by warp j: T_ij = -T_ii sum_m A_im T_mj, computed transposed
// (X_i = T_ij^T) so that a product's accumulators are the next one's left operand in registers.
constexpr int kPrepThreads = 128;
constexpr int kPrepLd = 68;   // row of the fp32 matrices, padded

template <int kD>
struct PrepCfg {
  static constexpr int kLd = kD + 8;   // row of K and Q, padded
  static constexpr uint32_t kRows = 2 * kChunk * kLd * 2;
  static constexpr uint32_t kUnion = kRows > 2 * kImgHalf ? kRows : 2 * kImgHalf;   // K, Q; then the image
  static constexpr uint32_t kMat = kChunk * kPrepLd * 4;
  static constexpr uint32_t kSmemBytes = kUnion + 2 * kMat + kChunk * 8 + kChunk * 4 + 16 + 128;
};

template <int kD>
__global__ void __launch_bounds__(kPrepThreads) litela_delta_prep(const DeltaArgs a, uint8_t* __restrict__ prep) {
  using namespace sm100;
  using Cfg = PrepCfg<kD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  __nv_bfloat16* Ks = reinterpret_cast<__nv_bfloat16*>(smem);
  __nv_bfloat16* Qs = Ks + kChunk * Cfg::kLd;
  uint8_t* image = smem;
  float* As = reinterpret_cast<float*>(smem + Cfg::kUnion);
  float* Tt = As + kChunk * kPrepLd;                 // T transposed: Tt[column][row]
  double* G = reinterpret_cast<double*>(Tt + kChunk * kPrepLd);
  float* beta = reinterpret_cast<float*>(G + kChunk);
  int* bad = reinterpret_cast<int*>(beta + kChunk);

  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, gr = lane >> 2, t2 = (lane & 3) * 2;
  pdl_launch_dependents();   // the chain waits for this grid before it reads what it wrote
  const int h = blockIdx.x % a.Hv, hk = h / (a.Hv / a.Hk);
  const long long slot = blockIdx.x / a.Hv;
  int s, n0;
  DeltaSeq sq;
  if (!delta_find(a, slot, lane, s, sq, n0)) return;
  const int len = min(kChunk, sq.len - n0);

  for (int i = tid; i < 2 * kChunk * (kD / 8); i += kPrepThreads) {
    const int c = i % (kD / 8), r = (i / (kD / 8)) % kChunk, m = i / (kChunk * (kD / 8));
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (r < len) x = *reinterpret_cast<const uint4*>(delta_row(m ? a.q : a.k, sq, n0 + r, hk) + c * 8);
    *reinterpret_cast<uint4*>((m ? Qs : Ks) + r * Cfg::kLd + c * 8) = x;
  }
  if (w == 0) {   // G, two tokens a lane
    double x[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = 2 * lane + j;
      x[j] = n < len ? (double)clamp_decay(a.g[sq.entry * a.g_sb + (long long)(sq.first + n0 + n) * a.g_st + h]) : 0.0;
    }
    x[1] += x[0];
    double run = x[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    const double before = run - x[1];
    G[2 * lane] = before + x[0];
    G[2 * lane + 1] = run;
  } else if (w < 3) {
    const int n = tid - 32;
    beta[n] = n < len ? a.beta[sq.entry * a.b_sb + (long long)(sq.first + n0 + n) * a.b_st + h] : 0.f;
  } else if (tid == 96) {
    *bad = kChunk;
  }
  __syncthreads();

  // K K^T and Q K^T, the warp's 16 rows, columns up to its diagonal block
  float accA[8][4], P[8][4];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) accA[n][i] = P[n][i] = 0.f;
  {
    const uint32_t* kr = reinterpret_cast<const uint32_t*>(Ks + (16 * w + gr) * Cfg::kLd + t2);
    const uint32_t* qr = reinterpret_cast<const uint32_t*>(Qs + (16 * w + gr) * Cfg::kLd + t2);
    const uint32_t* br = reinterpret_cast<const uint32_t*>(Ks + gr * Cfg::kLd + t2);
    constexpr int kW = Cfg::kLd / 2;   // a row in words
#pragma unroll
    for (int ks = 0; ks < kD / 16; ++ks) {
      const uint32_t ka[4] = {kr[ks * 8], kr[8 * kW + ks * 8], kr[ks * 8 + 4], kr[8 * kW + ks * 8 + 4]};
      const uint32_t qa[4] = {qr[ks * 8], qr[8 * kW + ks * 8], qr[ks * 8 + 4], qr[8 * kW + ks * 8 + 4]};
#pragma unroll
      for (int n = 0; n < 8; ++n)
        if (n < 2 * w + 2) {
          const uint32_t b[2] = {br[n * 8 * kW + ks * 8], br[n * 8 * kW + ks * 8 + 4]};
          mma_16816(accA[n], ka, b);
          mma_16816(P[n], qa, b);
        }
    }
  }
#pragma unroll
  for (int n = 0; n < 8; ++n)
    if (n < 2 * w + 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 16 * w + gr + (i >> 1) * 8, c = 8 * n + t2 + (i & 1);
        const float D = c <= r ? expf((float)(G[r] - G[c])) : 0.f;
        accA[n][i] = c < r ? beta[r] * accA[n][i] * D : 0.f;
        P[n][i] = c <= r ? P[n][i] * (a.scale * D) : 0.f;
        if (!isfinite(accA[n][i]) || !isfinite(P[n][i])) {
          accA[n][i] = P[n][i] = 0.f;
          atomicMin(bad, r);
        }
      }
      float* dst = As + (16 * w + gr) * kPrepLd + 8 * n + t2;
      *reinterpret_cast<float2*>(dst) = make_float2(accA[n][0], accA[n][1]);
      *reinterpret_cast<float2*>(dst + 8 * kPrepLd) = make_float2(accA[n][2], accA[n][3]);
    }
  __syncwarp();

  // the diagonal block: lane j solves for column j, x_i = delta_ij - sum_m<i A_im x_m
  if (lane < 16) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == lane ? 1.f : 0.f;
      const float* row = As + (16 * w + i) * kPrepLd + 16 * w;
#pragma unroll
      for (int m = 0; m < i; ++m) v -= row[m] * x[m];
      x[i] = v;
    }
    float4* dst = reinterpret_cast<float4*>(Tt + (16 * w + lane) * kPrepLd + 16 * w);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
  __syncthreads();

  // the blocks below it, block column w
  if (w < 3) {
    uint32_t xh[3][4], xl[3][4];   // X_m of the rows m = w + slot
#pragma unroll
    for (int e = 0; e < 3; ++e) {
      const int i = w + 1 + e;   // T's block row that this step makes
      if (i < 4) {
        if (e == 0) {
          float c[2][4];
          const float* src = Tt + (16 * w + gr) * kPrepLd + 16 * w + t2;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int q = 0; q < 4; ++q) c[n][q] = src[(q >> 1) * 8 * kPrepLd + 8 * n + (q & 1)];
          split_frag(c, xh[0], xl[0]);
        }
        float r[2][4] = {};
#pragma unroll
        for (int m = 0; m <= e; ++m) {   // sum over T's block rows w + m
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float* src = As + (16 * i + 8 * n + gr) * kPrepLd + 16 * (w + m) + t2;
            uint32_t bh[2], bl[2];
            split_bf16(src[0], src[1], bh[0], bl[0]);
            split_bf16(src[8], src[9], bh[1], bl[1]);
            mma_split(r[n], xh[m], xl[m], bh, bl);
          }
        }
        uint32_t rh[4], rl[4];
        split_frag(r, rh, rl);
        float x[2][4] = {};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float* src = Tt + (16 * i + t2) * kPrepLd + 16 * i + 8 * n + gr;   // T_ii[n][k] = Tt[k][n]
          uint32_t bh[2], bl[2];
          split_bf16(src[0], src[kPrepLd], bh[0], bl[0]);
          split_bf16(src[8 * kPrepLd], src[9 * kPrepLd], bh[1], bl[1]);
          mma_split(x[n], rh, rl, bh, bl);
#pragma unroll
          for (int q = 0; q < 4; ++q) x[n][q] = -x[n][q];
          float* dst = Tt + (16 * w + gr) * kPrepLd + 16 * i + 8 * n + t2;
          *reinterpret_cast<float2*>(dst) = make_float2(x[n][0], x[n][1]);
          *reinterpret_cast<float2*>(dst + 8 * kPrepLd) = make_float2(x[n][2], x[n][3]);
        }
        if (e < 2) split_frag(x, xh[e + 1], xl[e + 1]);
      }
    }
  }
  __syncthreads();

  // T into the image (K and Q are no longer needed), thread = row, 8 columns at a time
  for (int i = tid; i < kChunk * 8; i += kPrepThreads) {
    const int row = i & 63, c0 = (i >> 6) * 8;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = c0 + 2 * q;
      const float x0 = c <= row ? Tt[c * kPrepLd + row] : 0.f, x1 = c + 1 <= row ? Tt[(c + 1) * kPrepLd + row] : 0.f;
      split_bf16(x0, x1, hi[q], lo[q]);
    }
    *reinterpret_cast<uint4*>(image + sw128(row, c0)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(image + kImgHalf + sw128(row, c0)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  // P T, the warp's rows: sum over the blocks k up to its diagonal one, T's columns up to block k
  {
    float acc[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k <= w) {
        uint32_t ph[4], pl[4];
        split_frag(&P[2 * k], ph, pl);
#pragma unroll
        for (int n = 0; n < 8; ++n)
          if (n < 2 * k + 2) {
            const float* src = Tt + (8 * n + gr) * kPrepLd + 16 * k + t2;
            // inside the diagonal block Tt holds T's zeros above the diagonal
            uint32_t bh[2], bl[2];
            split_bf16(src[0], src[1], bh[0], bl[0]);
            split_bf16(src[8], src[9], bh[1], bl[1]);
            mma_split(acc[n], ph, pl, bh, bl);
          }
      }
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t hi, lo;
        split_bf16(acc[n][2 * r], acc[n][2 * r + 1], hi, lo);
        const uint32_t o = sw128(kChunk + 16 * w + gr + 8 * r, 8 * n + t2);
        *reinterpret_cast<uint32_t*>(image + o) = hi;
        *reinterpret_cast<uint32_t*>(image + kImgHalf + o) = lo;
      }
  }
  uint8_t* dst = prep + (slot * a.Hv + h) * (long long)kPrepBytes;
  float* fac = reinterpret_cast<float*>(dst + kPrepFactors);
  if (tid < kChunk) {
    const double end = G[len - 1];
    fac[kFacDecay + tid] = expf((float)G[tid]);
    fac[kFacToEnd + tid] = tid < len ? expf((float)(end - G[tid])) : 0.f;
    fac[kFacBeta + tid] = beta[tid];
    if (tid == 0) {
      fac[kFacChunk] = expf((float)end);
      reinterpret_cast<int*>(fac)[kFacBad] = *bad;
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    bulk_store(dst, image, 2 * kImgHalf);
    bulk_commit_group();
    bulk_wait_group<0>();
  }
}

// ---------------------------------------------------------------------------------------
// litela_delta_chain: one CTA walks the chunks of one sequence and value head for kCols of the
// state's columns (columns do not meet, so a state is cut by columns over CTAs).
//
// Three tcgen05 products per chunk, each with M = 128 rows, fp32 accumulators in TMEM:
//     X1 = [K; Q] S0           (rows: 64 of K, 64 of Q; K dimension d)
//     X2 = [T; P T] R          (K dimension 64)
//     X3 = K^T (e^(G_C - G) U) (rows: d; K dimension 64)
// Between them eight warps take the accumulators to registers, form R, then U, then the new state,
// and write them as bf16 pairs into shared memory as the next product's B operand.  The chain of
// these six steps is what a chunk costs; the loads of the next chunks, the output rows' arithmetic
// and their stores run beside it.  All B operands are tiles of 128-byte rows (row: K index, 64 bf16 columns,
// MN-major): with kCols = 64 a hi and a lo tile; with kCols = 32 one tile with hi and lo side by
// side, whose products land in two column ranges that the readers add.
//
// Warps: 0-7 accumulators (warp % 4: TMEM lanes; warp / 4: which half of the columns), 8 issues
// the products, 9-12 load (cp.async for the strided K, Q, V rows; one bulk copy for the prepared
// block).  Every wait is bounded; a time-out is recorded in *err.
constexpr int kChainStages = 2;
constexpr int kChainThreads = 13 * 32;
constexpr int kLoadThreads = 4 * 32;
constexpr uint32_t kChainTmem = 256;
enum : int { kErrChainLoad = 0x510, kErrChainMma = 0x520, kErrChainAcc = 0x530 };

template <int kD, int kCols>
struct ChainCfg {
  static constexpr int kBlocks = kD > 64 ? 2 : 1;                 // 64-channel blocks of K and Q
  static constexpr uint32_t kKQ = kBlocks * 16384;                // per block: 64 rows of K, 64 of Q
  static constexpr uint32_t kVLd = kCols * 2 + 16;                // padded row of V
  static constexpr uint32_t kV = 64 * kVLd;
  static constexpr uint32_t kOffPrep = kKQ;
  static constexpr uint32_t kOffV = kKQ + kPrepBytes;
  static constexpr uint32_t kStage = (kOffV + kV + 1023) / 1024 * 1024;
  static constexpr int kTiles = kCols == 64 ? 2 : 1;              // tiles of a B operand
  static constexpr uint32_t kSTile = kD * 128, kRTile = 64 * 128;
  static constexpr uint32_t kOffS = kChainStages * kStage;
  static constexpr uint32_t kOffR = kOffS + kTiles * kSTile;
  static constexpr uint32_t kOffBars = kOffR + kTiles * kRTile;
  static constexpr uint32_t kSmemBytes = kOffBars + 256 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory above the 227 KB per-block limit");
};

// kN accumulators of this thread's TMEM lane from column c of a product's 64 columns
template <int kCols, int kN>
__device__ __forceinline__ void chain_acc(uint32_t taddr, int c, float* x) {
  using namespace sm100;
  if (kCols == 64) {
    uint32_t r[32];
    tmem_ld_x32(taddr + c, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = __uint_as_float(r[i]);
  } else {   // the hi and the lo operand's columns
    uint32_t r[16], l[16];
    tmem_ld_x16(taddr + c, r);
    tmem_ld_x16(taddr + 32 + c, l);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = __uint_as_float(r[i]) + __uint_as_float(l[i]);
  }
}

// kN values of a B operand's row, columns c .. c + kN - 1, as a bf16 pair
template <int kCols, int kN>
__device__ __forceinline__ void chain_put(uint8_t* tile, uint32_t lo_tile, int row, int c, const float* x) {
#pragma unroll
  for (int i = 0; i < kN; i += 8) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) split_bf16(x[i + 2 * q], x[i + 2 * q + 1], hi[q], lo[q]);
    *reinterpret_cast<uint4*>(tile + sw128(row, c + i)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(kCols == 64 ? tile + lo_tile + sw128(row, c + i) : tile + sw128(row, 32 + c + i)) =
        make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

template <int kD, int kCols>
__global__ void __launch_bounds__(kChainThreads, 1)
litela_delta_chain(const DeltaArgs a, const uint8_t* __restrict__ prep, int* __restrict__ err) {
  using namespace sm100;
  using Cfg = ChainCfg<kD, kCols>;
  constexpr int kN = kCols / 2;   // columns of an accumulator warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stile = smem + Cfg::kOffS;
  uint8_t* rtile = smem + Cfg::kOffR;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);   // K, Q, V rows landed
  uint64_t* pfull = full + kChainStages;                                // the prepared block landed
  uint64_t* empty = pfull + kChainStages;
  uint64_t* done = empty + kChainStages;   // X1, X2, X3
  uint64_t* sready = done + 3;
  uint64_t* rready = sready + 1;
  uint64_t* uready = rready + 1;
  uint64_t* drained = uready + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* first_bad = reinterpret_cast<int*>(tmem_holder + 2);   // first token whose R was not finite

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kParts = kD / kCols;
  const int part = blockIdx.x % kParts, h = (blockIdx.x / kParts) % a.Hv, s = blockIdx.x / (kParts * a.Hv);
  const int hk = h / (a.Hv / a.Hk);
  const DeltaSeq sq = delta_seq(a, s);
  const int nchunk = (sq.len + kChunk - 1) / kChunk;
  const uint8_t* blocks = prep + (delta_slot0(a, s, sq) * a.Hv + h) * (long long)kPrepBytes;
  const long long block_step = (long long)a.Hv * kPrepBytes;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kChainStages; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&pfull[i], 1);
      mbar_init(&empty[i], 9);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&done[i], 1);
    mbar_init(sready, 8);
    mbar_init(rready, 4);
    mbar_init(uready, 4);
    mbar_init(drained, 1);
    *abort_flag = 0;
    *first_bad = 0x7fffffff;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_holder, kChainTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;

  if (warp < 8) {
    const int quad = warp & 3, c0 = (warp >> 2) * kN, row = quad * 32 + lane;
    const uint32_t ta = tmem + ((uint32_t)(quad * 32) << 16);
    const bool has_state = row < kD;       // this thread has a row of the state
    const bool is_q = quad >= 2;           // ... of the first two products: a row of Q, else of K
    const int tok = row & 63;
    const long long sbase = ((long long)s * a.Hv + h) * (kD * kD) + (long long)row * kD + part * kCols + c0;
    float S[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) S[i] = 0.f;
    if (has_state && a.state_in != nullptr)
#pragma unroll
      for (int i = 0; i < kN; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(a.state_in + sbase + i);
        S[i] = x.x, S[i + 1] = x.y, S[i + 2] = x.z, S[i + 3] = x.w;
      }
    bool ok = true;
    auto hand = [&](uint64_t* bar) {   // this warp's shared-memory writes and TMEM reads are done
      fence_proxy_async_smem();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto wait = [&](uint64_t* bar, int phase, int code) {
      ok = ok && mbar_wait(bar, phase & 1, abort_flag, err, kErrChainAcc | code);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after_sync();
      return ok;
    };
    if (nchunk > 0) {
      if (has_state) chain_put<kCols, kN>(stile, Cfg::kSTile, row, c0, S);
      hand(sready);
    }
    for (int n = 0; n < nchunk; ++n) {
      const int st = n % kChainStages;
      uint8_t* stage = smem + st * Cfg::kStage;
      if (!wait(&full[st], n / kChainStages, 0) || !wait(&pfull[st], n / kChainStages, 1)) break;
      const float* fac = reinterpret_cast<const float*>(stage + Cfg::kOffPrep + kPrepFactors);
      const float decay = fac[kFacDecay + tok], to_end = fac[kFacToEnd + tok], beta = fac[kFacBeta + tok];
      const float chunk_decay = fac[kFacChunk];
      const int prep_bad = reinterpret_cast<const int*>(fac)[kFacBad];
      uint4 v[kN / 8];
      if (!is_q)
#pragma unroll
        for (int i = 0; i < kN / 8; ++i)
          v[i] = *reinterpret_cast<const uint4*>(stage + Cfg::kOffV + tok * Cfg::kVLd + c0 * 2 + i * 16);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      float x[kN];
      if (!wait(&done[0], n, 2)) break;
      if (!is_q) {   // R = beta (v - e^G K S0)
        chain_acc<kCols, kN>(ta, c0, x);
        float zero = 0.f;   // stays 0 while all are finite
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const uint32_t wv = reinterpret_cast<const uint32_t*>(v)[i / 2];
          x[i] = beta * (__uint_as_float((i & 1) ? wv & 0xFFFF0000u : wv << 16) - decay * x[i]);
          zero += 0.f * x[i];
        }
        if (zero != 0.f) {
#pragma unroll
          for (int i = 0; i < kN; ++i) x[i] = 0.f;
          atomicMin(first_bad, n * kChunk + tok);
        }
        chain_put<kCols, kN>(rtile, Cfg::kRTile, tok, c0, x);
        hand(rready);
      } else {       // the output's share of S0
        chain_acc<kCols, kN>(ta, c0, x);
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] *= a.scale * decay;
      }
      if (!wait(&done[1], n, 3)) break;
      const bool bad = tok >= prep_bad || n * kChunk + tok >= *static_cast<volatile int*>(first_bad);
      const float nan = __int_as_float(0x7fffffff);
      if (!is_q) {   // e^(G_C - G) U
        chain_acc<kCols, kN>(ta + 64, c0, x);
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = bad ? nan : x[i] * to_end;
        chain_put<kCols, kN>(rtile, Cfg::kRTile, tok, c0, x);
        hand(uready);
      } else {
        float y[kN];
        chain_acc<kCols, kN>(ta + 64, c0, y);
#pragma unroll
        for (int i = 0; i < kN; ++i) y[i] = bad ? nan : y[i] + x[i];
        if (n * kChunk + tok < sq.len) {
          uint4* o = reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(delta_row(a.out, sq, n * kChunk + tok, h)) +
                                              part * kCols + c0);
#pragma unroll
          for (int i = 0; i < kN; i += 8)
            o[i / 8] = make_uint4(pack_bf16(y[i], y[i + 1]), pack_bf16(y[i + 2], y[i + 3]),
                                  pack_bf16(y[i + 4], y[i + 5]), pack_bf16(y[i + 6], y[i + 7]));
        }
      }
      if (!wait(&done[2], n, 4)) break;
      if (has_state) {   // (a warp's 32 rows are all of the state, or none)
        chain_acc<kCols, kN>(ta + 128, c0, x);
#pragma unroll
        for (int i = 0; i < kN; ++i) S[i] = chunk_decay * S[i] + x[i];
        if (n + 1 < nchunk) chain_put<kCols, kN>(stile, Cfg::kSTile, row, c0, S);
      }
      if (n + 1 < nchunk) hand(sready);
    }
    if (ok && has_state && a.state_out != nullptr)
#pragma unroll
      for (int i = 0; i < kN; i += 4)
        *reinterpret_cast<float4*>(a.state_out + sbase + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
  } else if (warp == 8) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, 64, false, true);
      constexpr uint32_t idesc_t = idesc_bf16_f32(128, 64, true, true);
      const uint32_t sa = smem_u32(stile), ra = smem_u32(rtile);
      auto wait = [&](uint64_t* bar, int phase, int code) {
        const bool ok = mbar_wait(bar, phase & 1, abort_flag, err, kErrChainMma | code);
        tc_fence_after_sync();
        return ok;
      };
      for (int n = 0; n < nchunk; ++n) {
        const int st = n % kChainStages;
        const uint32_t kq = smem_u32(smem + st * Cfg::kStage), img = kq + Cfg::kOffPrep;
        if (!wait(&full[st], n / kChainStages, 0) || !wait(sready, n, 1)) break;
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks) {
          const uint64_t ad = smem_desc(kq + (ks / 4) * 16384 + (ks % 4) * 32, 16, 1024, kSwizzle128B);
#pragma unroll
          for (int t = 0; t < Cfg::kTiles; ++t)
            umma_bf16(tmem, ad, smem_desc(sa + t * Cfg::kSTile + ks * 2048, 1024, 1024, kSwizzle128B), idesc, ks | t);
        }
        umma_commit(&done[0]);
        if (!wait(&pfull[st], n / kChainStages, 2) || !wait(rready, n, 3)) break;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint64_t hi = smem_desc(img + ks * 32, 16, 1024, kSwizzle128B);
          const uint64_t lo = smem_desc(img + kImgHalf + ks * 32, 16, 1024, kSwizzle128B);
          const uint64_t b = smem_desc(ra + ks * 2048, 1024, 1024, kSwizzle128B);
          umma_bf16(tmem + 64, hi, b, idesc, ks);
          if (Cfg::kTiles == 2)
            umma_bf16(tmem + 64, hi, smem_desc(ra + Cfg::kRTile + ks * 2048, 1024, 1024, kSwizzle128B), idesc, 1u);
          umma_bf16(tmem + 64, lo, b, idesc, 1u);
        }
        umma_commit(&done[1]);
        if (!wait(uready, n, 4)) break;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          // K^T: M over channels.  d = 128: the second 64 are the next block.  Smaller d: rows 64
          // on take Q's channels, results that nobody reads.
          const uint64_t ad = smem_desc(kq + ks * 2048, kD > 64 ? 16384 : 8192, 1024, kSwizzle128B);
#pragma unroll
          for (int t = 0; t < Cfg::kTiles; ++t)
            umma_bf16(tmem + 128, ad, smem_desc(ra + t * Cfg::kRTile + ks * 2048, 1024, 1024, kSwizzle128B), idesc_t,
                      ks | t);
        }
        umma_commit(&done[2]);
        umma_commit(&empty[st]);
      }
      // products in flight end before the memory under them is given back
      umma_commit(drained);
      mbar_drain(drained, 0);
    }
  } else {
    const int t = threadIdx.x - 9 * 32;
    pdl_wait_primary();
    fence_proxy_async_global();   // the prepared blocks are read by bulk copies
    int issued = 0;
    for (int n = 0; n < nchunk; ++n) {
      const int st = n % kChainStages;
      bool ok = n < kChainStages ||
                mbar_wait(&empty[st], (n / kChainStages - 1) & 1, abort_flag, err, kErrChainLoad | st);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint8_t* stage = smem + st * Cfg::kStage;
      if (t == 0) {
        mbar_arrive_expect_tx(&pfull[st], kPrepBytes);
        bulk_load(stage + Cfg::kOffPrep, blocks + n * block_step, kPrepBytes, &pfull[st]);
      }
      issued = n + 1;
      const int n0 = n * kChunk, len = min(kChunk, sq.len - n0);
      const uint32_t kq = smem_u32(stage), vs = kq + Cfg::kOffV;
#pragma unroll 4
      for (int i = t; i < 128 * (kD / 8); i += kLoadThreads) {
        const int c = i % (kD / 8), r = i / (kD / 8);   // row: 64 of K, then 64 of Q
        const int tok = r & 63;
        const bool real = tok < len;
        const __nv_bfloat16* src = delta_row(r < 64 ? a.k : a.q, sq, n0 + (real ? tok : 0), hk) + c * 8;
        cp_async_16(kq + (c / 8) * 16384 + sw128(r, (c % 8) * 8), src, real);
      }
#pragma unroll 4
      for (int i = t; i < 64 * (kCols / 8); i += kLoadThreads) {
        const int c = i % (kCols / 8), tok = i / (kCols / 8);
        const bool real = tok < len;
        cp_async_16(vs + tok * Cfg::kVLd + c * 16, delta_row(a.v, sq, n0 + (real ? tok : 0), h) + part * kCols + c * 8,
                    real);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
    }
    if (t == 0 && *abort_flag)   // bulk copies still in flight land before the CTA exits
      for (int i = issued > kChainStages ? issued - kChainStages : 0; i < issued; ++i)
        mbar_drain(&pfull[i % kChainStages], (i / kChainStages) & 1);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kChainTmem);
  }
}

}  // namespace litela
