// The gated delta rule over whole sequences, in chunks of 64 tokens.
//
// With G_i the sum of the log decays of a chunk's tokens up to i, S0 the state before the chunk,
// D_ij = e^(G_i - G_j) for i >= j, and the chunk's rows as matrices K, Q, V [64, d]:
//     L = K K^T . D below the diagonal,               P = scale (Q K^T . D),
//     E = V - diag(e^G) K S0                          (what the state before the chunk gets wrong)
//     W = (I + L diag(beta))^-1 E                     (what the state before each token gets wrong)
//     U = diag(beta) W                                (the written values)
//     out = scale diag(e^G) Q S0 + P U,               S = e^G_C S0 + K^T diag(e^(G_C - G)) U.
// With T = (I + diag(beta) L)^-1 and X = L T (both need no state):
//     W = E - X R,   P U = P T R,   R = diag(beta) E.
// litela_delta_prep makes X and P T for all chunks at once.  What is left of a chunk are three
// products that follow one another, and litela_delta_chain walks a sequence's chunks with them.
// (X rather than T: the unit diagonal's share of W stays in fp32 registers, and W is there for the
// gradient of beta, where beta may be 0.)
//
// Precision.  States are fp32 and stay in registers.  An fp32 operand of a tensor-core product is
// entered in three bf16 terms (each the rounding of what the ones before it leave: 2^-9, 2^-17 and 2^-25
// relative), all products of terms that reach 2^-25 of the first, summed in fp32: states are 1 to 3e-7 off
// against 64 bits, as with plain fp32 operations.  With two terms of X, P T and of the blocks that X is made of
// they were up to 2e-6 off (d = 32); the third costs the blocks a fifth to a quarter (16384 tokens, 32 heads of 128: 209 ->
// 249 us) and the chain 6 % (532 -> 564).  K, Q and V are bf16 already.  G is summed in fp64: differences
// of large sums of decays would lose in fp32.
//
// A NaN or an infinity must not reach the tokens before its own: 0 * NaN inside a product would
// carry it there.  So non-finite entries are taken out of L, P, beta and R, the first token that had one
// is kept, and it and all later tokens of the sequence (and the state) get NaN.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>

#include "f32x2.cuh"
#include "litela_delta.cuh"
#include "sm100_ptx.cuh"

namespace litela {

constexpr int kChunk = 64;

// One chunk and value head's prepared block: X^T and (P T)^T as images of tcgen05 A operands (MN-major:
// 64 rows x 128 columns bf16 in two blocks of 64 columns, 128-byte swizzle), one image for each of
// the three bf16 terms, then per-token factors.  The columns (the product's rows, TMEM lanes) hold 16 rows
// of X, the same 16 rows of P T, the next 16 rows of X and so on, as do the rows of K and Q in the
// chain's tile: every warp's quarter of the lanes then has 16 tokens of either kind.
constexpr uint32_t kImgTerm = 128 * 128;   // one of them
__host__ __device__ constexpr int lane_of(int token) { return 32 * (token / 16) + token % 16; }
constexpr uint32_t kPrepFactors = 3 * kImgTerm;
constexpr uint32_t kFactorBytes = 2304;
constexpr uint32_t kPrepBytes = kPrepFactors + kFactorBytes;
// A training step's block has a second image behind it, X and P T not transposed: rows are tokens i,
// columns as above for tokens j, (i, j) of X and of P T (the gradient's products take X^T and (P T)^T)
constexpr uint32_t kPrepSaveBytes = kPrepBytes + 3 * kImgTerm;
// fp32 at kPrepFactors: e^G [64], e^(G_C - G) [64] (0 behind the end), beta [64] (0 behind the
// end), then e^G_C and (int32) the first token of the chunk with a non-finite L, P or beta, or 64
constexpr int kFacDecay = 0, kFacToEnd = 64, kFacBeta = 128, kFacChunk = 192, kFacBad = 193;
// and what D is made of (litela_delta_prep): e^(G_r - G_m) [64]; e^(G_m - G_c) for the blocks of rows
// 1, 2, 3 (48 each, from kFacCol + 48 on); G_r - G_m in two fp32 terms [64][2]
constexpr int kFacRow = 196, kFacCol = kFacRow + 64 - 48, kFacRel = kFacCol + 192;
static_assert((kFacRel + 128) * 4 <= kFactorBytes, "factors");

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
__device__ __forceinline__ bool delta_find(const DeltaArgs& a, int slot, int lane, int& s, DeltaSeq& q, int& n0) {
  if (a.cu == nullptr) {
    const int nc = (a.ntok + kChunk - 1) / kChunk;
    s = slot / nc;
    q = delta_seq(a, s);
    n0 = (slot - s * nc) * kChunk;
    return true;
  }
  int lo = 0, hi = a.nseq;   // the last s with cu[s] / 64 + s <= slot is in [lo, hi)
  while (true) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool below = at < hi && min(max(a.cu[at], 0), a.ntok) / kChunk + at <= slot;
    const int n = __popc(__ballot_sync(0xffffffffu, below));
    if (n == 0) return false;
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) break;
  }
  s = lo;
  q = delta_seq(a, s);
  n0 = (slot - (int)delta_slot0(a, s, q)) * kChunk;
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
// the next bf16 term of a pair, which it leaves
__device__ __forceinline__ uint32_t next_term(F2& y, bool last) {
  const float2 z = f2_out(y);
  const uint32_t w = pack_bf16(z.x, z.y);
  if (!last) y = f2_fma(f2_bf16(w), f2(-1.f, -1.f), y);
  return w;
}
// (a, b) in three terms, w[0], w[step], w[2 step]
__device__ __forceinline__ void split_terms(float a, float b, uint32_t* w, int step) {
  F2 y = f2(a, b);
#pragma unroll
  for (int t = 0; t < 3; ++t) w[t * step] = next_term(y, t == 2);
}
// 16 x 16 accumulators (two 16 x 8 tiles) as an A operand in three terms
__device__ __forceinline__ void split_frag(const float (*c)[4], uint32_t (*a)[4]) {
  split_terms(c[0][0], c[0][1], &a[0][0], 4);
  split_terms(c[0][2], c[0][3], &a[0][1], 4);
  split_terms(c[1][0], c[1][1], &a[0][2], 4);
  split_terms(c[1][2], c[1][3], &a[0][3], 4);
}
// byte offset of bf16 element (row, column < 64) in a tile of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t sw128(int row, int col) {
  return (uint32_t)(row * 128 + ((((col >> 3) ^ row) & 7) << 4) + (col & 7) * 2);
}

// ---------------------------------------------------------------------------------------
// litela_delta_prep: X and P T of one chunk and value head per CTA, transposed (the image).
//
// mma.sync: the operands are one chunk's, 64 rows, and X is made of 16 x 16 blocks where each
// product waits for the one before; a tcgen05 product would be a sixth full and go through TMEM and
// shared memory for each block.
//   1. K and Q by cp.async; G, and D's factors.  With m the first row of r's block of 16 and c
//      before it, D_rc = e^(G_r - G_m) e^(G_m - G_c): 160 exponentials instead of 1536, both
//      factors at most 1.
//   2. K K^T and Q K^T up to the diagonal, to shared memory in fp32; there D makes them L and P.
//   3. X's diagonal blocks by substitution, one lane a column: x_i = L_ij - sum_m<i L_im beta_m x_m.
//   4. The blocks below them, block column j by one warp:
//      X_ij = (I - X_ii diag(beta)) (L_ij - sum_m L_im diag(beta) X_mj),
//      computed transposed, so that a product's accumulators are the next one's left operand in
//      registers.  X^T takes the places above L's diagonal, which are free.
//   5. P T = P - (P diag(beta)) X.
//   6. The images' terms, from X's fp32 values and P T's accumulators.
// Operands are fp32 in shared memory (as much as two bf16 terms would take) and cut into three terms in
// registers.
// A chunk is a chain of latencies, a fetch of instructions being one of them: a CTA runs through its
// code once.  So loops stay rolled, and three CTAs an SM overlap.
constexpr int kPrepThreads = 256;
constexpr int kPrepLd = 68;   // row of L and P in fp32, padded
constexpr uint32_t kImgBlock = 64 * 128;   // half of the columns of an image, one bf16 term
// byte offset in the image of (row, token of X); of P T: 32 bytes on, before the swizzle
__device__ __forceinline__ uint32_t img_off(int row, int token, int is_p) {
  const int m = lane_of(token) + 16 * is_p;
  return (m >> 6) * kImgBlock + sw128(row, m & 63);
}

template <int kD>
struct PrepCfg {
  static constexpr int kLd = kD + 8;   // row of K and Q, padded
  static constexpr uint32_t kRows = 2 * kChunk * kLd * 2;
  static constexpr uint32_t kUnion = kRows > 2 * kImgTerm ? kRows : 2 * kImgTerm;   // K, Q; then the image
  static constexpr uint32_t kOffL = kUnion;                                  // L, fp32
  static constexpr uint32_t kOffP = kOffL + kChunk * kPrepLd * 4;
  static constexpr uint32_t kOffG = kOffP + kChunk * kPrepLd * 4;
  static constexpr uint32_t kOffBeta = kOffG + kChunk * 8;
  static constexpr uint32_t kOffRow = kOffBeta + kChunk * 4;                 // e^(G_r - G_m)
  static constexpr uint32_t kOffCol = kOffRow + kChunk * 4;                  // e^(G_m - G_c), by block of r
  static constexpr uint32_t kOffRel = kOffCol + 4 * 48 * 4;                  // G_r - G_m, two fp32 terms
  static constexpr uint32_t kOffBad = kOffRel + kChunk * 8;
  static constexpr uint32_t kSmemBytes = kOffBad + 16 + 128;
  static_assert(3 * (kSmemBytes + 1024) <= 228 * 1024, "three CTAs an SM");
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, const uint32_t* r) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void stmatrix_x2(uint32_t addr, uint32_t r0, uint32_t r1) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(r0), "r"(r1) : "memory");
}
__device__ __forceinline__ void stmatrix_x2_t(uint32_t addr, uint32_t r0, uint32_t r1) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(r0), "r"(r1) : "memory");
}
__device__ __forceinline__ void stmatrix_x4_t(uint32_t addr, const uint32_t* r) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// d[n] + small[n] += A B[n], fp32 operands in three terms each, all products that reach 2^-25 of the first;
// two accumulators, so that a product waits for every other one before it only
template <int kTiles>
__device__ __forceinline__ void mma_terms(float (*d)[4], float (*small)[4], const uint32_t (*a)[4], const uint32_t (*b)[3][2]) {
  auto all = [&](float (*to)[4], int ta, int tb) {
#pragma unroll
    for (int n = 0; n < kTiles; ++n) sm100::mma_16816(to[n], a[ta], b[n][tb]);
  };
  all(small, 2, 0), all(d, 1, 0), all(small, 1, 1), all(d, 0, 1), all(small, 0, 2), all(d, 0, 0);
}
// a B operand tile (16 x 8) in three terms: B[k][n] = src[n * kPrepLd + k]
__device__ __forceinline__ void prep_tile(const float* src, int lane, uint32_t (*b)[2]) {
  const float* p = src + (lane >> 2) * kPrepLd + (lane & 3) * 2;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 v = *reinterpret_cast<const float2*>(p + 8 * i);
    split_terms(v.x, v.y, &b[0][i], 2);
  }
}

template <int kD, bool kSave>
__global__ void __launch_bounds__(kPrepThreads, 3) litela_delta_prep(const DeltaArgs a, uint8_t* __restrict__ prep) {
  using namespace sm100;
  using Cfg = PrepCfg<kD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  float* Lf = reinterpret_cast<float*>(smem + Cfg::kOffL);   // L; X^T with and above its diagonal
  float* Pf = reinterpret_cast<float*>(smem + Cfg::kOffP);
  // the image's terms, the third one in P's place
  auto image = [&](int t) { return t < 2 ? smem + t * kImgTerm : smem + Cfg::kOffP; };
  double* G = reinterpret_cast<double*>(smem + Cfg::kOffG);
  float* beta = reinterpret_cast<float*>(smem + Cfg::kOffBeta);
  float* rowf = reinterpret_cast<float*>(smem + Cfg::kOffRow);
  float* colf = reinterpret_cast<float*>(smem + Cfg::kOffCol);
  float2* rel = reinterpret_cast<float2*>(smem + Cfg::kOffRel);
  int* bad = reinterpret_cast<int*>(smem + Cfg::kOffBad);

  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, gr = lane >> 2, t2 = (lane & 3) * 2;
  pdl_launch_dependents();   // the chain waits for this grid before it reads what it wrote
  const int slot = blockIdx.x / a.Hv, h = blockIdx.x - slot * a.Hv, hk = h / (a.Hv / a.Hk);
  if (a.zero_rest) delta_zero_rest(a, a.out, a.Hv, kD);
  int s, n0;
  DeltaSeq sq;
  if (!delta_find(a, slot, lane, s, sq, n0)) return;
  const int len = min(kChunk, sq.len - n0);

  double g0[2] = {0.0, 0.0};   // two tokens a lane
  if (w == 0) {
    const float* g = a.g + sq.entry * a.g_sb + (long long)(sq.first + n0) * a.g_st + h;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (2 * lane + j < len) g0[j] = (double)clamp_decay(g[(2 * lane + j) * a.g_st]);
  }
  {   // a thread copies one 16-byte column of every kStep-th row
    constexpr int kC = kD / 8, kStep = kPrepThreads / kC;
    const int c = tid % kC, r0 = tid / kC;
    const __nv_bfloat16* kp = delta_row(a.k, sq, n0 + r0, hk) + c * 8;
    const __nv_bfloat16* qp = delta_row(a.q, sq, n0 + r0, hk) + c * 8;
    const long long ks = kStep * a.k.st, qs = kStep * a.q.st;
    const uint32_t dst = smem_u32(smem) + r0 * (Cfg::kLd * 2) + c * 16;
#pragma unroll
    for (int i = 0; i < kChunk / kStep; ++i) {
      const bool real = r0 + i * kStep < len;
      cp_async_16(dst + i * kStep * (Cfg::kLd * 2), real ? kp : a.k.p, real);
      cp_async_16(dst + (kChunk + i * kStep) * (Cfg::kLd * 2), real ? qp : a.q.p, real);
      kp += ks;
      qp += qs;
    }
    cp_async_commit();
  }
  bool bad_beta = false;
  if (w == 0) {
    double run = g0[0] + g0[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    const double before = __shfl_up_sync(0xffffffffu, run, 1);   // (not run - g0[1]: that may be NaN - NaN)
    G[2 * lane] = (lane == 0 ? 0.0 : before) + g0[0];
    G[2 * lane + 1] = run;
  } else if (w < 3) {
    const int n = tid - 32;
    const float b = n < len ? a.beta[sq.entry * a.b_sb + (long long)(sq.first + n0 + n) * a.b_st + h] : 0.f;
    // 0 for the products, in which zeros stand for earlier tokens; the token is kept as a bad one
    bad_beta = !isfinite(b);
    beta[n] = bad_beta ? 0.f : b;
  } else if (tid == 96) {
    *bad = kChunk;
  }
  __syncthreads();
  if (bad_beta) atomicMin(bad, tid - 32);
  uint8_t* dst = prep + ((long long)slot * a.Hv + h) * (kSave ? kPrepSaveBytes : kPrepBytes);
  float* fac = reinterpret_cast<float*>(dst + kPrepFactors);
  if (tid < kChunk) {
    const double d = G[tid] - G[tid & ~15];
    rel[tid] = make_float2((float)d, (float)(d - (double)(float)d));
    rowf[tid] = expf((float)d);
    fac[kFacRow + tid] = rowf[tid];
    *reinterpret_cast<float2*>(fac + kFacRel + 2 * tid) = rel[tid];
  } else if (tid < kChunk + 96) {   // blocks 1, 2, 3 of r have 16, 32, 48 columns before them
    const int i = tid - kChunk, b = i < 16 ? 1 : i < 48 ? 2 : 3, c = i - (b == 1 ? 0 : b == 2 ? 16 : 48);
    fac[kFacCol + b * 48 + c] = colf[b * 48 + c] = expf((float)(G[16 * b] - G[c]));
  } else if (tid >= 192) {   // the chain's factors
    const int n = tid - 192;
    const double end = G[len - 1];
    fac[kFacDecay + n] = expf((float)G[n]);
    fac[kFacToEnd + n] = n < len ? expf((float)(end - G[n])) : 0.f;
    fac[kFacBeta + n] = beta[n];
    if (n == 0) fac[kFacChunk] = expf((float)end);
  }
  cp_async_wait<0>();
  __syncthreads();

  {   // K K^T (even warps) and Q K^T (odd ones): rows 16 rb .., the 2 rb + 2 tiles of 8 columns
    const int rb = w >> 1, is_p = w & 1;
    float acc[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    const uint32_t base = smem_u32(smem);
    const uint32_t aa = base + (is_p * kChunk + 16 * rb + (lane & 15)) * (Cfg::kLd * 2) + (lane >> 4) * 16;
    const uint32_t ba = base + (lane & 7) * (Cfg::kLd * 2) + (lane >> 3) * 16;
#pragma unroll 1
    for (int ks = 0; ks < kD / 32; ++ks) {   // 32 channels
      uint32_t a0[4], a1[4];
      ldmatrix_x4(a0, aa + ks * 64);
      ldmatrix_x4(a1, aa + ks * 64 + 32);
#pragma unroll
      for (int m = 0; m < 8; m += 4)
        if (m < 2 * rb + 2) {   // four tiles (the last ones may lie right of the diagonal block)
          uint32_t b[4][4];
#pragma unroll
          for (int n = 0; n < 4; ++n) ldmatrix_x4(b[n], ba + (m + n) * 8 * (Cfg::kLd * 2) + ks * 64);
#pragma unroll
          for (int n = 0; n < 4; ++n) mma_16816(acc[m + n], a0, b[n]);
#pragma unroll
          for (int n = 0; n < 4; ++n) mma_16816(acc[m + n], a1, b[n] + 2);
        }
    }
    float* dst = (is_p ? Pf : Lf) + (16 * rb + gr) * kPrepLd + t2;
#pragma unroll
    for (int n = 0; n < 8; ++n)
      if (n < 2 * rb + 2) {
        *reinterpret_cast<float2*>(dst + 8 * n) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2*>(dst + 8 * kPrepLd + 8 * n) = make_float2(acc[n][2], acc[n][3]);
      }
  }
  __syncthreads();   // K and Q are done with: the image takes their place
  // D makes them L and P: a thread has 4 columns of every block of 16 up to the diagonal one of a row
  int first = kChunk;
  {
    const int r = tid >> 2, c0 = (tid & 3) * 4, rb = r >> 4;
    const float rf = rowf[r];
    const float2 rr = rel[r];
    const float4* cf = reinterpret_cast<const float4*>(colf + rb * 48 + c0);
    float4 *ls = reinterpret_cast<float4*>(Lf + r * kPrepLd + c0), *ps = reinterpret_cast<float4*>(Pf + r * kPrepLd + c0);
    auto scaled = [&](float4* src, const float* f, int real = 4) {   // the first `real` columns, zeros
      const float4 x = *src;
      float4 y = make_float4(real > 0 ? x.x * f[0] : 0.f, real > 1 ? x.y * f[1] : 0.f, real > 2 ? x.z * f[2] : 0.f,
                             real > 3 ? x.w * f[3] : 0.f);
      if (0.f * y.x + 0.f * y.y + 0.f * y.z + 0.f * y.w != 0.f) {   // not finite
        first = min(first, r);
        y.x = isfinite(y.x) ? y.x : 0.f, y.y = isfinite(y.y) ? y.y : 0.f;
        y.z = isfinite(y.z) ? y.z : 0.f, y.w = isfinite(y.w) ? y.w : 0.f;
      }
      return y;
    };
#pragma unroll 1
    for (int cb = 0; cb < rb; ++cb) {
      const float4 c4 = cf[4 * cb];
      float f[4] = {rf * c4.x, rf * c4.y, rf * c4.z, rf * c4.w};
      ls[4 * cb] = scaled(ls + 4 * cb, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] *= a.scale;
      ps[4 * cb] = scaled(ps + 4 * cb, f);
    }
    float f[4];   // the diagonal block: L below the diagonal, P with it (what f is above it is not used)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 rc = rel[16 * rb + c0 + e];
      f[e] = expf((rr.x - rc.x) + (rr.y - rc.y));
    }
    const int below = r - 16 * rb - c0;   // columns of the four that are left of the diagonal
    ls[4 * rb] = scaled(ls + 4 * rb, f, below);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] *= a.scale;
    ps[4 * rb] = scaled(ps + 4 * rb, f, below + 1);
  }
  if (first < kChunk) atomicMin(bad, first);
  __syncthreads();

  // X's diagonal block w: lane j solves for column j; it takes L's place, transposed
  if (w < 4 && lane < 16) {
    float x[16], bx[16];
    float* blk = Lf + 16 * w * kPrepLd + 16 * w;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v[4] = {blk[i * kPrepLd + lane], 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 l = *reinterpret_cast<const float4*>(blk + i * kPrepLd + m);
        v[0] -= l.x * bx[m];
        if (m + 1 < i) v[1] -= l.y * bx[m + 1];
        if (m + 2 < i) v[2] -= l.z * bx[m + 2];
        if (m + 3 < i) v[3] -= l.w * bx[m + 3];
      }
      x[i] = i > lane ? (v[0] + v[1]) + (v[2] + v[3]) : 0.f;
      bx[i] = beta[16 * w + i] * x[i];
    }
    __syncwarp(0xffffu);
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<float4*>(blk + lane * kPrepLd + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  }
  __syncthreads();

  // the blocks below them, block column w; X_iw goes to the free block (w, i), transposed
  if (w < 3) {
    uint32_t y[3][3][4];   // -(diag(beta) X)^T of the block rows w, w + 1, w + 2 (zero: not made yet), by term
#pragma unroll
    for (int m = 1; m < 3; ++m)
#pragma unroll
      for (int q = 0; q < 12; ++q) y[m][q / 4][q % 4] = 0u;
    float* own = Lf + (16 * w + gr) * kPrepLd + t2;   // rows of X^T: 8 q; columns: 16 times a block, 8 n
    {
      float v[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = 16 * w + 8 * n;
          const float2 x = *reinterpret_cast<const float2*>(own + 8 * q * kPrepLd + i);
          v[n][2 * q] = -beta[i + t2] * x.x;
          v[n][2 * q + 1] = -beta[i + t2 + 1] * x.y;
        }
      split_frag(v, y[0]);
    }
#pragma unroll 1
    for (int i = w + 1; i < 4; ++i) {   // X's block row i
      float x[2][4], xs[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)   // L_iw transposed
          xs[n][e] = 0.f, x[n][e] = Lf[(16 * i + 8 * n + t2 + (e & 1)) * kPrepLd + 16 * w + gr + 8 * (e >> 1)];
#pragma unroll
      for (int m = 0; m < 3; ++m)   // sum over X's block rows w + m before i
        if (w + m < i) {
          uint32_t b[2][3][2];
#pragma unroll
          for (int n = 0; n < 2; ++n) prep_tile(Lf + (16 * i + 8 * n) * kPrepLd + 16 * (w + m), lane, b[n]);
          mma_terms<2>(x, xs, y[m], b);
        }
      float br[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          x[n][q] += xs[n][q], xs[n][q] = 0.f;
          br[n][q] = -beta[16 * i + 8 * n + t2 + (q & 1)] * x[n][q];
        }
      uint32_t r[3][4], b[2][3][2];
      split_frag(br, r);
#pragma unroll
      for (int n = 0; n < 2; ++n)   // X_ii^T stands as rows of the K dimension
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* v = Lf + (16 * i + t2 + 8 * h) * kPrepLd + 16 * i + 8 * n + gr;
          split_terms(v[0], v[kPrepLd], &b[n][0][h], 2);
        }
      mma_terms<2>(x, xs, r, b);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          x[n][2 * q] += xs[n][2 * q], x[n][2 * q + 1] += xs[n][2 * q + 1];
          *reinterpret_cast<float2*>(own + 8 * q * kPrepLd + 16 * i + 8 * n) = make_float2(x[n][2 * q], x[n][2 * q + 1]);
          x[n][2 * q] *= -beta[16 * i + 8 * n + t2];
          x[n][2 * q + 1] *= -beta[16 * i + 8 * n + t2 + 1];
        }
      split_frag(x, r);
#pragma unroll
      for (int m = 1; m < 3; ++m)
        if (i == w + m)
#pragma unroll
          for (int q = 0; q < 12; ++q) y[m][q / 4][q % 4] = r[q / 4][q % 4];
    }
  }
  __syncthreads();

  // P T = P - (P diag(beta)) X in blocks (row, column) of 16 x 16, row - column + 1 products each: a
  // warp has one block, the last two warps have two on the diagonal (2 blocks apart); four products at most
  constexpr uint32_t kBlockRow = 0x10321323u, kBlockCol = 0x10210100u;   // by warp, 4 bits each
  const int rb0 = kBlockRow >> (4 * w) & 15, cb0 = kBlockCol >> (4 * w) & 15, blocks = w < 6 ? 1 : 2;
  float acc[2][2][4];
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (u < blocks) {
      const int rb = rb0 + 2 * u, cb = cb0 + 2 * u;
      const float* prow = Pf + (16 * rb + gr) * kPrepLd + t2;
      float small[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 v = *reinterpret_cast<const float2*>(prow + 8 * q * kPrepLd + 16 * cb + 8 * n);
          acc[u][n][2 * q] = v.x, acc[u][n][2 * q + 1] = v.y;
          small[n][2 * q] = small[n][2 * q + 1] = 0.f;
        }
#pragma unroll 1
      for (int k = cb; k <= rb; ++k) {
        uint32_t p[3][4], b[2][3][2];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = 16 * k + (q >> 1) * 8;
          const float2 v = *reinterpret_cast<const float2*>(prow + (q & 1) * 8 * kPrepLd + c);
          const float2 bc = *reinterpret_cast<const float2*>(beta + c + t2);
          split_terms(-bc.x * v.x, -bc.y * v.y, &p[0][q], 4);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) prep_tile(Lf + (16 * cb + 8 * e) * kPrepLd + 16 * k, lane, b[e]);
        mma_terms<2>(acc[u], small, p, b);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[u][n][q] += small[n][q];
    }
  __syncthreads();   // P has been read

  // An image's three terms into shared memory: X's from its fp32 values, P T's from the accumulators.
  // kSecond: not transposed (a training step's)
  const int l8 = lane & 7, k8 = ((lane >> 3) & 1) * 8;
  auto write_image = [&](auto second) {
    constexpr bool kSecond = decltype(second)::value;
#pragma unroll 1
    for (int i = tid; i < kChunk * 8; i += kPrepThreads) {   // a row and 8 of its columns
      const int row = i & 63, c0 = (i >> 6) * 8;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
      if (kSecond ? (c0 >> 4) <= (row >> 4) : (c0 >> 4) >= (row >> 4))
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = kSecond ? Lf[(c0 + e) * kPrepLd + row] : Lf[row * kPrepLd + c0 + e];
      uint32_t t[3][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) split_terms(v[2 * q], v[2 * q + 1], &t[0][q], 4);
#pragma unroll
      for (int h = 0; h < 3; ++h)
        *reinterpret_cast<uint4*>(image(h) + img_off(row, c0, 0)) = make_uint4(t[h][0], t[h][1], t[h][2], t[h][3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i / 2 < blocks) {   // matrices by lane / 8: the first term of rows 0..7 and 8..15, the second
        const float* x = acc[i / 2][i % 2];
        uint32_t v[3][2];
        split_terms(x[0], x[1], &v[0][0], 2);
        split_terms(x[2], x[3], &v[0][1], 2);
        const int r = 16 * (rb0 + i / 2 * 2), c = 16 * (cb0 + i / 2 * 2) + 8 * (i % 2);
        const uint32_t o = kSecond ? img_off(r + k8 + l8, c, 1) : img_off(c + l8, r + k8, 1);
        const uint32_t first = smem_u32(image(lane >> 4)) + o, third = smem_u32(image(2)) + o;
        if (kSecond) {
          stmatrix_x4(first, &v[0][0]);
          stmatrix_x2(third, v[2][0], v[2][1]);
        } else {
          stmatrix_x4_t(first, &v[0][0]);
          stmatrix_x2_t(third, v[2][0], v[2][1]);
        }
      }
    // the blocks of (P T)^T left of its diagonal blocks are zero (of P T, right of them): six of 16 rows x 32 bytes
    if (tid < 192) {
      const int blk = tid >> 5, hi = blk < 1 ? 1 : blk < 3 ? 2 : 3, lo = blk - (hi == 1 ? 0 : hi == 2 ? 1 : 3);
      const uint32_t o = img_off(16 * (kSecond ? lo : hi) + ((lane >> 1) & 15), 16 * (kSecond ? hi : lo) + (lane & 1) * 8, 1);
#pragma unroll
      for (int h = 0; h < 3; ++h) *reinterpret_cast<uint4*>(image(h) + o) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      uint8_t* to = dst + (kSecond ? kPrepBytes : 0u);
      bulk_store(to, image(0), 2 * kImgTerm);
      bulk_store(to + 2 * kImgTerm, image(2), kImgTerm);
      bulk_commit_group();
      bulk_wait_group_read<0>();
    }
  };
  if (tid == 0) reinterpret_cast<int*>(dst + kPrepFactors)[kFacBad] = *bad;
  write_image(std::false_type{});
  if constexpr (kSave) {
    __syncthreads();   // (the first image has been taken)
    write_image(std::true_type{});
  }
}

// ---------------------------------------------------------------------------------------
// litela_delta_chain: one CTA walks the chunks of one sequence and value head for 32 of the state's
// columns (columns do not meet, so a state is cut by columns over CTAs): 2.2 us a chunk at d = 128.  64
// columns a CTA took 3.2 us a chunk where 32 took 2.0 to 2.2: less for many equal sequences (1.6 a half), but a
// long sequence among others, or few heads, wait for the longest chain of chunks.
//
// Three tcgen05 products per chunk, each with M = 128 rows, fp32 accumulators in TMEM:
//     X1 = [K; Q] S0           (rows: 16 of K, 16 of Q, 16 of K ..; K dimension d)
//     X2 = [X; P T] R          (rows alike; K dimension 64)
//     X3 = K^T (e^(G_C - G) U) (rows: d; K dimension 64)
// Between them eight warps take the accumulators to registers, form E and R, then W and U, then the
// new state, and write them in bf16 terms into shared memory as the next product's B operand.  The
// chain of these six steps is what a chunk costs; the loads of the next chunks, the output rows'
// arithmetic and their stores run beside it.  All B operands are tiles of 128-byte rows (row: K index,
// 64 bf16 columns, MN-major), two terms of 32 columns side by side in a tile, whose products land in
// column ranges of their own that the readers add.
//
// Warps: 0-7 accumulators (warp % 4: TMEM lanes; warp / 4: which half of the columns), 8 and 9 load
// (cp.async for the strided K, Q, V rows; one bulk copy for the prepared block), 10 issues the
// products.  The accumulator warps hand over with named barriers (one-way ~40 cycles; an mbarrier wait
// costs ~170 here even when its phase is over), the tensor core with mbarriers; waits for loads stand
// where a warp would idle anyway.  A tcgen05 product of 16 of the K dimension takes ~47 cycles whatever
// N <= 96 is (its operands' shared-memory bytes), so terms go side by side where that saves products.
// Every mbarrier wait is bounded; after a time-out (recorded in *err) all roles run their loops to
// the end without waiting, so that the named barriers stay matched.
constexpr int kCols = 32;   // of the state, a CTA's
constexpr int kChainStages = 2;
constexpr int kAccWarps = 8;
constexpr int kIssueWarp = kAccWarps + 2;   // on a scheduler whose accumulator warps have rows of Q
constexpr int kLoadWarps = 2;
constexpr int kChainThreads = (kAccWarps + 1 + kLoadWarps) * 32;   // 11 warps: up to 168 registers a thread
constexpr int kLoadThreads = kLoadWarps * 32;
constexpr uint32_t kChainTmem = 512;
enum : int { kErrChainLoad = 0x510, kErrChainMma = 0x520, kErrChainAcc = 0x530 };
// named barriers: S0, R and U are in shared memory (accumulator warps arrive, the issuer waits)
enum : int { kBarS = 1, kBarR = 2, kBarU = 3 };
constexpr int kBarThreads = (kAccWarps + 1) * 32;

// a shared-memory descriptor in halves: an offset of n bytes adds n / 16 to the lower one
struct Desc {
  uint32_t lo, hi;
};
__device__ __forceinline__ Desc desc_halves(uint32_t saddr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  const uint64_t d = sm100::smem_desc(saddr, lbo, sbo, swizzle);
  return Desc{(uint32_t)d, (uint32_t)(d >> 32)};
}
__device__ __forceinline__ Desc operator+(Desc d, uint32_t n) { return Desc{d.lo + n, d.hi}; }
__device__ __forceinline__ void umma(uint32_t d_tmem, Desc a, Desc b, uint32_t idesc, uint32_t accumulate) {
  sm100::umma_bf16(d_tmem, a.lo, a.hi, b.lo, b.hi, idesc, accumulate);
}

template <int kD>
struct ChainCfg {
  static constexpr int kBlocks = kD > 64 ? 2 : 1;                 // 64-channel blocks of K and Q
  static constexpr uint32_t kKQ = kBlocks * 16384;                // per block: 64 rows of K and of Q
  static constexpr uint32_t kVLd = kCols * 2 + 16;                // padded row of V
  static constexpr uint32_t kV = 64 * kVLd;
  static constexpr uint32_t kOffPrep = kKQ;
  static constexpr uint32_t kOffV = kKQ + kPrepBytes;
  static constexpr uint32_t kStage = (kOffV + kV + 1023) / 1024 * 1024;
  static constexpr uint32_t kSTile = kD * 128;                    // S0 (three terms, two tiles)
  static constexpr uint32_t kRTile = 64 * 128;                    // R and U (three terms, two tiles)
  static constexpr uint32_t kOffS = kChainStages * kStage;
  static constexpr uint32_t kOffR = kOffS + 2 * kSTile;
  static constexpr uint32_t kOffBars = kOffR + 2 * kRTile;
  static constexpr uint32_t kX1 = 0, kX2 = 96, kX3 = 192;         // TMEM columns of the three products
  static constexpr uint32_t kSmemBytes = kOffBars + 256 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory above the 227 KB per-block limit");
  static_assert(kLoadThreads == kChunk, "a loading thread prefetches one row");
};

// A warp's share of a product whose B operand has kTerms terms, 16 columns from c on (all of one kind: fp32 pairs).
// chain_acc: its 32 lanes, a lane's columns to its thread.  chain_frag: 16 of its lanes: thread t gets
// the rows t / 4 and t / 4 + 8, columns 2 (t % 4) of each 8, as x[2 g + half].
constexpr int kN = kCols * 4 / kAccWarps;   // columns of an accumulator warp
static_assert(kN == 16, "an accumulator warp has 16 columns");
template <int kTerms>
__device__ __forceinline__ void add_terms(const uint32_t (*r)[kN], F2* x) {
  auto get = [&](int t, int i) { return f2(__uint_as_float(r[t][2 * i]), __uint_as_float(r[t][2 * i + 1])); };
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) {   // the small terms first
    x[i] = get(kTerms - 1, i);
#pragma unroll
    for (int t = kTerms - 2; t >= 0; --t) x[i] = f2_add(x[i], get(t, i));
  }
}
template <int kTerms>
__device__ __forceinline__ void chain_acc(uint32_t taddr, int c, F2* x) {
  uint32_t r[kTerms][kN];
#pragma unroll
  for (int t = 0; t < kTerms; ++t) sm100::tmem_ld_x16(taddr + 32 * t + c, r[t]);
  sm100::tmem_wait_ld();
  add_terms<kTerms>(r, x);
}
template <int kTerms>
__device__ __forceinline__ void chain_frag(uint32_t taddr, int c, F2* x) {
  uint32_t r[kTerms][kN / 2];
#pragma unroll
  for (int t = 0; t < kTerms; ++t) sm100::tmem_ld_16x256b_x2(taddr + 32 * t + c, r[t]);
  sm100::tmem_wait_ld();
  auto get = [&](int t, int i) { return f2(__uint_as_float(r[t][2 * i]), __uint_as_float(r[t][2 * i + 1])); };
#pragma unroll
  for (int i = 0; i < kN / 4; ++i) {
    x[i] = get(kTerms - 1, i);
#pragma unroll
    for (int t = kTerms - 2; t >= 0; --t) x[i] = f2_add(x[i], get(t, i));
  }
}

// Into a B operand's tiles: the thread's kN values (pairs) of a row, columns c .. c + kN - 1, in kTerms
// bf16 terms
template <int kTerms>
__device__ __forceinline__ void chain_put(uint8_t* tile, uint32_t tile_bytes, int row, int c, const F2* x) {
#pragma unroll
  for (int i = 0; i < kN; i += 8) {
    F2 y[4] = {x[i / 2], x[i / 2 + 1], x[i / 2 + 2], x[i / 2 + 3]};
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = next_term(y[q], t + 1 == kTerms);
      *reinterpret_cast<uint4*>(tile + (t / 2) * tile_bytes + sw128(row, (t & 1) * 32 + c + i)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}
// ... a thread's part of chain_frag's arrangement; row: of its first half, c: its first column; the
// first term goes to the tiles' columns 32 kFirst on
template <int kTerms, int kFirst = 0>
__device__ __forceinline__ void chain_put_frag(uint8_t* tile, uint32_t tile_bytes, int row, int c, const F2* x) {
#pragma unroll
  for (int i = 0; i < kN / 4; ++i) {
    F2 y = x[i];
    const int r = row + (i & 1) * 8, cc = c + (i >> 1) * 8;
#pragma unroll
    for (int t = 0; t < kTerms; ++t)
      *reinterpret_cast<uint32_t*>(tile + ((t + kFirst) / 2) * tile_bytes + sw128(r, ((t + kFirst) & 1) * 32 + cc)) =
          next_term(y, t + 1 == kTerms);
  }
}

// What a training step's forward leaves for its backward, per chunk slot and value head: S0 as the B
// operand tiles of the chain (for each 32 columns twice d rows x 128 bytes: two terms, the third), and
// W in fp32 [64, d].
struct DeltaSaved {
  uint8_t* states;
  float* w;
};

template <int kD, bool kSave>
__global__ void __launch_bounds__(kChainThreads, 1)
litela_delta_chain(const DeltaArgs a, const uint8_t* __restrict__ prep, const DeltaSaved saved, int* __restrict__ err) {
  using namespace sm100;
  using Cfg = ChainCfg<kD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stile = smem + Cfg::kOffS;
  uint8_t* rtile = smem + Cfg::kOffR;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);   // K, Q, V and the block landed
  uint64_t* empty = full + kChainStages;
  uint64_t* done = empty + kChainStages;   // X1, X2, X3
  uint64_t* drained = done + 3;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* first_bad = reinterpret_cast<int*>(tmem_holder + 2);   // first token whose R was not finite

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kParts = kD / kCols;
  const int part = blockIdx.x % kParts, h = (blockIdx.x / kParts) % a.Hv, s = blockIdx.x / (kParts * a.Hv);
  const int hk = h / (a.Hv / a.Hk);
  const DeltaSeq sq = delta_seq(a, s);
  const int nchunk = (sq.len + kChunk - 1) / kChunk;
  const long long slot0 = delta_slot0(a, s, sq);
  constexpr long long kBlock = kSave ? kPrepSaveBytes : kPrepBytes;
  const uint8_t* blocks = prep + (slot0 * a.Hv + h) * kBlock;
  const long long block_step = a.Hv * kBlock;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kChainStages; ++i) {
      mbar_init(&full[i], kLoadWarps + 1);
      mbar_init(&empty[i], kAccWarps + 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&done[i], 1);
    mbar_init(drained, 1);
    *abort_flag = 0;
    *first_bad = 0x7fffffff;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_holder, kChainTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;

  if (warp < kAccWarps) {
    const int quad = warp & 3, c0 = (warp >> 2) * kN, row = quad * 32 + lane;
    const uint32_t ta = tmem + ((uint32_t)(quad * 32) << 16), tq = ta + (16u << 16);   // lanes of K's, of Q's rows
    const bool has_state = row < kD;                                 // this thread has a row of the state
    const int tok = quad * 16 + (lane >> 2), fc = c0 + (lane & 3) * 2;   // chain_frag: tokens tok and tok + 8
    const long long sbase = ((long long)s * a.Hv + h) * (kD * kD) + (long long)row * kD + part * kCols + c0;
    F2 S[kN / 2];
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) S[i] = f2(0.f, 0.f);
    if (has_state && a.state_in != nullptr)
#pragma unroll
      for (int i = 0; i < kN; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(a.state_in + sbase + i);
        S[i / 2] = f2(x.x, x.y), S[i / 2 + 1] = f2(x.z, x.w);
      }
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase, int code) {
      if (ok) ok = mbar_wait(bar, phase & 1, abort_flag, err, kErrChainAcc | code);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after_sync();
    };
    auto hand = [&](int id, int count) {   // this warp's shared-memory writes and TMEM reads are done
      fence_proxy_async_smem();
      tc_fence_before_sync();
      bar_arrive(id, count);
    };
    float decay[2] = {}, to_end[2] = {}, beta[2] = {}, chunk_decay = 0.f;
    int prep_bad = 0;
    uint32_t v[kN / 4];
    auto fetch = [&](int n) {   // chunk n's factors and values
      const int st = n % kChainStages;
      const uint8_t* stage = smem + st * Cfg::kStage;
      wait(&full[st], n / kChainStages, 0);
      const float* fac = reinterpret_cast<const float*>(stage + Cfg::kOffPrep + kPrepFactors);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        decay[i] = fac[kFacDecay + tok + 8 * i];
        to_end[i] = fac[kFacToEnd + tok + 8 * i];
        beta[i] = fac[kFacBeta + tok + 8 * i];
      }
      chunk_decay = fac[kFacChunk];
      prep_bad = reinterpret_cast<const int*>(fac)[kFacBad];
#pragma unroll
      for (int i = 0; i < kN / 4; ++i)
        v[i] = *reinterpret_cast<const uint32_t*>(stage + Cfg::kOffV + (tok + (i & 1) * 8) * Cfg::kVLd + (fc + (i >> 1) * 8) * 2);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    };
    if (nchunk > 0) {
      if (has_state) chain_put<3>(stile, Cfg::kSTile, row, c0, S);
      hand(kBarS, kBarThreads);
    }
    for (int n = 0; n < nchunk; ++n) {
      fetch(n);   // while the first product runs
      F2 e[kN / 4], x[kN / 2], y[kN / 4];
      wait(&done[0], n, 2);
      // E = v - e^G K S0, R = beta E
      chain_frag<3>(ta + Cfg::kX1, c0, e);
      F2 zero = f2(0.f, 0.f);   // stays 0 while all are finite
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const float d = decay[i & 1], b = beta[i & 1];
        e[i] = f2_fma(f2(-d, -d), e[i], f2_bf16(v[i]));
        x[i] = f2_mul(f2(b, b), e[i]);
        zero = f2_fma(f2(0.f, 0.f), x[i], zero);
      }
      const float2 z = f2_out(zero);
      if (z.x + z.y != 0.f) {
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) {
          const float2 xi = f2_out(x[i]);
          const bool fx = isfinite(xi.x), fy = isfinite(xi.y);
          if (!fx || !fy) atomicMin(first_bad, n * kChunk + tok + (i & 1) * 8);
          x[i] = f2(fx ? xi.x : 0.f, fy ? xi.y : 0.f);   // (the others may be an earlier token's)
        }
      }
      chain_put_frag<3>(rtile, Cfg::kRTile, tok, fc, x);
      hand(kBarR, kBarThreads);
      chain_frag<3>(tq + Cfg::kX1, c0, y);   // the output's share of S0
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const float d = a.scale * decay[i & 1];
        y[i] = f2_mul(f2(d, d), y[i]);
      }
      wait(&done[1], n, 3);
      const int bad_from = min(prep_bad, *static_cast<volatile int*>(first_bad) - n * kChunk);
      const float nan = __int_as_float(0x7fffffff);
      // W = E - X R, e^(G_C - G) U = e^(G_C - G) beta W
      chain_frag<3>(ta + Cfg::kX2, c0, x);
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const float f = tok + (i & 1) * 8 >= bad_from ? nan : to_end[i & 1] * beta[i & 1];
        e[i] = f2_fma(f2(-1.f, -1.f), x[i], e[i]);
        x[i] = f2_mul(f2(f, f), e[i]);
      }
      chain_put_frag<3>(rtile, Cfg::kRTile, tok, fc, x);
      hand(kBarU, kBarThreads);
      if constexpr (kSave) {
        float* w = saved.w + ((slot0 + n) * a.Hv + h) * (long long)(kChunk * kD) + part * kCols + fc;
#pragma unroll
        for (int i = 0; i < kN / 4; ++i)
          *reinterpret_cast<float2*>(w + (tok + (i & 1) * 8) * kD + (i >> 1) * 8) =
              tok + (i & 1) * 8 >= bad_from ? make_float2(nan, nan) : f2_out(e[i]);
      }
      // the output, while the third product runs
      chain_frag<3>(tq + Cfg::kX2, c0, x);
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const int t = tok + (i & 1) * 8;
        const float2 o = f2_out(f2_add(x[i], y[i]));
        if (n * kChunk + t < sq.len)
          *reinterpret_cast<uint32_t*>(const_cast<__nv_bfloat16*>(delta_row(a.out, sq, n * kChunk + t, h)) + part * kCols +
                                       fc + (i >> 1) * 8) = t >= bad_from ? 0x7fff7fffu : pack_bf16(o.x, o.y);
      }
      wait(&done[2], n, 4);
      if (has_state) {   // (a warp's 32 rows are all of the state, or none)
        chain_acc<3>(ta + Cfg::kX3, c0, x);
        const F2 d2 = f2(chunk_decay, chunk_decay);
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) S[i] = f2_fma(d2, S[i], x[i]);
        if (n + 1 < nchunk) chain_put<3>(stile, Cfg::kSTile, row, c0, S);
      }
      if (n + 1 < nchunk) hand(kBarS, kBarThreads);
    }
    if (ok && has_state && a.state_out != nullptr)
#pragma unroll
      for (int i = 0; i < kN; i += 4)
        *reinterpret_cast<float4*>(a.state_out + sbase + i) =
            make_float4(f2_out(S[i / 2]).x, f2_out(S[i / 2]).y, f2_out(S[i / 2 + 1]).x, f2_out(S[i / 2 + 1]).y);
  } else if (warp == kIssueWarp) {
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 96, false, true);
    constexpr uint32_t idesc_r = idesc_bf16_f32(128, 96, true, true);    // three terms
    constexpr uint32_t idesc_2 = idesc_bf16_f32(128, 64, true, true);    // two terms
    constexpr uint32_t idesc_1 = idesc_bf16_f32(128, 32, true, true);    // one
    // descriptors of each operand's first 16 of the K dimension
    const Desc sdesc = desc_halves(smem_u32(stile), Cfg::kSTile, 1024, kSwizzle128B);
    const Desc rdesc = desc_halves(smem_u32(rtile), Cfg::kRTile, 1024, kSwizzle128B);
    const Desc kqdesc = desc_halves(smem_u32(smem), 16, 1024, kSwizzle128B);
    const Desc imgdesc = desc_halves(smem_u32(smem) + Cfg::kOffPrep, kImgBlock, 1024, kSwizzle128B);
    // K^T: M over channels, 16 tokens every 32 rows.  d = 128: the second 64 channels are the next
    // block.  Smaller d: rows 64 on take other rows, results that nobody reads.
    const Desc ktdesc = desc_halves(smem_u32(smem), kD > 64 ? 16384 : 8192, 1024, kSwizzle128B);
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase, int code) {
      if (ok && lane == 0) ok = mbar_spin(bar, phase & 1, abort_flag, err, kErrChainMma | code);
      ok = __all_sync(0xffffffffu, ok);
    };
    if (nchunk > 0) wait(&full[0], 0, 0);
    for (int n = 0; n < nchunk; ++n) {
      const int st = n % kChainStages;
      const uint32_t off = st * (Cfg::kStage / 16);
      bar_sync(kBarS, kBarThreads);
      tc_fence_after_sync();
      if (lane == 0) {
        if (kSave) {
          bulk_store(saved.states + (((slot0 + n) * a.Hv + h) * kParts + part) * (2LL * Cfg::kSTile), stile, 2 * Cfg::kSTile);
          bulk_commit_group();
        }
        if (ok) {
#pragma unroll
          for (int ks = 0; ks < kD / 16; ++ks)
            umma(tmem + Cfg::kX1, kqdesc + off + (ks / 4) * 1024 + (ks % 4) * 2, sdesc + ks * 128, idesc_s, ks > 0);
          umma_commit(&done[0]);
        }
      }
      __syncwarp();
      bar_sync(kBarR, kBarThreads);
      tc_fence_after_sync();
      if (ok && lane == 0) {
        // X's and P T's first term by all three of R, the second by two, the third by one
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma(tmem + Cfg::kX2, imgdesc + off + ks * 128, rdesc + ks * 128, idesc_r, ks > 0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma(tmem + Cfg::kX2, imgdesc + off + kImgTerm / 16 + ks * 128, rdesc + ks * 128, idesc_2, 1u);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma(tmem + Cfg::kX2, imgdesc + off + 2 * kImgTerm / 16 + ks * 128, rdesc + ks * 128, idesc_1, 1u);
        umma_commit(&done[1]);
      }
      __syncwarp();
      bar_sync(kBarU, kBarThreads);
      tc_fence_after_sync();
      if (lane == 0) {
        if (kSave) bulk_wait_group_read<0>();   // before the tile of S0 is written again
        if (ok) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma(tmem + Cfg::kX3, ktdesc + off + ks * 256, rdesc + ks * 128, idesc_r, ks > 0);
          umma_commit(&done[2]);
          umma_commit(&empty[st]);
        }
      }
      __syncwarp();
      // while the accumulator warps make the next S0
      if (n + 1 < nchunk) wait(&full[(n + 1) % kChainStages], (n + 1) / kChainStages, 0);
    }
    if (lane == 0) {   // products in flight end before the memory under them is given back
      umma_commit(drained);
      mbar_drain(drained, 0);
    }
  } else {
    const int t = threadIdx.x - (warp > kIssueWarp ? kAccWarps + 1 : kAccWarps) * 32;
    pdl_wait_primary();
    fence_proxy_async_global();   // the prepared blocks are read by bulk copies
    int issued = 0;
    // A thread copies one 16-byte column of every kStep-th row, of K and Q and of V: its places in a
    // stage differ by constants, its places in memory by a stride.
    constexpr int kC = kD / 8, kStep = kLoadThreads / kC, kVC = kCols / 8, kVStep = kLoadThreads / kVC;
    const int r0 = t / kC, c = t % kC, vr0 = t / kVC;
    const uint32_t kq0 = smem_u32(smem) + (c / 8) * 16384 + sw128(lane_of(r0), (c % 8) * 8);
    const uint32_t v0 = smem_u32(smem) + Cfg::kOffV + vr0 * Cfg::kVLd + (t % kVC) * 16;
    const __nv_bfloat16* kp = delta_row(a.k, sq, r0, hk) + c * 8;
    const __nv_bfloat16* qp = delta_row(a.q, sq, r0, hk) + c * 8;
    const __nv_bfloat16* vp = delta_row(a.v, sq, vr0, h) + part * kCols + (t % kVC) * 8;
    const long long kstep = kStep * a.k.st, qstep = kStep * a.q.st, vstep = kVStep * a.v.st;
    for (int n = 0; n < nchunk; ++n) {
      const int st = n % kChainStages;
      const bool ok = n < kChainStages || lane != 0 ||
                      mbar_wait(&empty[st], (n / kChainStages - 1) & 1, abort_flag, err, kErrChainLoad | st);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (t == 0) {
        mbar_arrive_expect_tx(&full[st], kPrepBytes);
        bulk_load(smem + st * Cfg::kStage + Cfg::kOffPrep, blocks + n * block_step, kPrepBytes, &full[st]);
      }
      issued = n + 1;
      const int n0 = n * kChunk, len = min(kChunk, sq.len - n0);
      const uint32_t dkq = kq0 + st * Cfg::kStage, dv = v0 + st * Cfg::kStage;
#pragma unroll
      for (int i = 0; i < kChunk / kStep; ++i) {
        // row r0 + i kStep (r0 < kStep, powers of two: the swizzle is r0's, xor the step's); Q's row is 16 on
        const uint32_t o = (dkq ^ (((i * kStep) & 7) << 4)) + lane_of(i * kStep) * 128;
        const bool real = r0 + i * kStep < len;
        cp_async_16(o, real ? kp : a.k.p, real);
        cp_async_16(o + 2048, real ? qp : a.q.p, real);
        kp += kstep;
        qp += qstep;
      }
#pragma unroll
      for (int i = 0; i < kChunk / kVStep; ++i) {
        const bool real = vr0 + i * kVStep < len;
        cp_async_16(dv + i * kVStep * Cfg::kVLd, real ? vp : a.v.p, real);
        vp += vstep;
      }
      if (n + 1 < nchunk) {   // the next chunk's rows and block into L2: their turn comes a chunk later
        const int r = n0 + kChunk + t;
        if (r < sq.len) {
          const __nv_bfloat16 *k = delta_row(a.k, sq, r, hk), *q = delta_row(a.q, sq, r, hk);
          prefetch_l2(k);
          prefetch_l2(q);
          if (kD > 64) {
            prefetch_l2(k + 64);
            prefetch_l2(q + 64);
          }
          prefetch_l2(delta_row(a.v, sq, r, h) + part * kCols);
        }
        if (t == 0) bulk_prefetch_l2(blocks + (n + 1) * block_step, kPrepBytes);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
    }
    if (t == 0 && *abort_flag)   // bulk copies still in flight land before the CTA exits
      for (int i = issued > kChainStages ? issued - kChainStages : 0; i < issued; ++i)
        mbar_drain(&full[i % kChainStages], (i / kChainStages) & 1);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kChainTmem);
  }
}

}  // namespace litela
