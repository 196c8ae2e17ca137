// Gradient of the gated delta rule over whole sequences, from what a forward kept (DeltaSaved and the
// prepared blocks).  Names as in litela_delta_chunk.cuh; do is the gradient of out, G' that of the
// state behind a chunk, dU that of the written values, and with w_i the gradient of what token i
// writes, before beta:
//     dU = P^T do + diag(e^(G_C - G)) K G',     w = T^T dU,     y = diag(beta) w,     dv = y,
//     G' (before the chunk) = e^G_C G' + scale Q^T diag(e^G) do - K^T diag(e^G) y,
//     dbeta_i = w_i . W_i
//     dq = scale diag(e^G) do S0^T + (M1 . D) K,            M1 = scale do U^T with and below the diagonal,
//     dk = (M1 . D)^T Q + diag(e^(G_C - G)) U G'^T - diag(e^G) y S0^T - (M2 . D) K - (M2 . D)^T K,
//                                                           M2 = y U^T below the diagonal,
// and, as the decay of token t is a factor of everything that goes from before t to t or later,
//     dg_t = e^G_C <S0, G'> + sum over i >= t of c_i + sum over j < t of b_j + sum over j < t <= i of N_ij,
//     N = (M1 . D) . Q K^T - (M2 . D) . K K^T,  c = the products of q and k with their terms of S0,
//                                               b = Z U, that of k with its term of G' (Z in litela_delta_back).
// The last sum is one over s >= t of N's row s less its column s.  (<S_C, G'> and the sums of
// q . dq - y . v are the same in exact arithmetic, but cancel where decays are strong, with the errors of
// bf16 pairs: dg 1.8e-5 off against 64 bits for 3 x 208 tokens, 4 heads of 32, where this form was 2e-6 off with
// pairs and is 3e-7 off now.)
//
// litela_delta_back walks a sequence's chunks from the last to the first (as litela_delta_chain, with
// the same three products a chunk) and leaves y and each chunk's G'; litela_delta_grads makes the rest,
// all chunks at once.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "litela_delta_chunk.cuh"

namespace litela {

struct DeltaGrads {
  DeltaView dout, dq, dk, dv;      // dq, dk: key heads
  float* dg;                       // [entry, token, Hv], dense
  float* dbeta;
  const float* dstate_out;         // [sequence][Hv][d][d] or null (zeros)
  float* dstate_in;                // or null
  // between the two kernels, per chunk slot and value head
  uint8_t* gstates;                // G', two terms, as the first tiles of DeltaSaved's states
  float* y;                        // [d / 32] tiles of 64 rows of 32 columns, placed by y_off
  float* rows;                     // [d / 32][2][2][64]: w . W and b of half of 32 columns
  float* ends;                     // [d / 32][8]: shares of <S0, G'>
};

// place of (row, column < 32) in a tile of y, in floats: 16-byte pieces of a row change places with the row, so
// that eight rows' equal columns lie in different banks
__device__ __forceinline__ int y_off(int row, int col) {
  return row * 32 + ((((col >> 2) ^ ((row & 3) << 1) ^ ((row >> 2) & 1)) & 7) << 2) + (col & 3);
}

__device__ __forceinline__ float sum_warp(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------------------------------
// litela_delta_back: one CTA walks the chunks of one sequence and value head for 32 columns of the
// state's gradient, as litela_delta_chain.  Per chunk, each product with M = 128 rows:
//     X1 = [K; Q] G'
//     X2 = [X; P T]^T [do, -diag(beta) Z],  Z = diag(e^(G_C - G)) K G'
//     X3 = [K; Q]^T [-diag(e^G) y; scale diag(e^G) do]
// Rows (TMEM lanes) of the first two alternate, 16 of K's or X's and 16 of Q's or P T's.  X1's rows of K
// are used, and of X2 the columns of Z in X's rows and the columns of do in P T's rows, which are the
// same tokens: w = Z + X2 (T = I - diag(beta) X) and G' = e^G_C G' + X3.  G', Z, y, X and P T in three terms
// as in litela_delta_chain: dbeta and dstate_in are 2 to 5e-7 off (with two of G', X and P T 1.8 to 2.7e-6
// and 0.9e-6; the third costs 4 %).  Bound by the chain of its steps: 3.4 us a chunk at d = 128 (2 x 2048
// tokens, 16 heads: 109 us).
template <int kD>
struct BackCfg {
  static constexpr int kBlocks = kD > 64 ? 2 : 1;
  static constexpr uint32_t kKQ = kBlocks * 16384;                // per block: 64 rows of K and of Q
  static constexpr uint32_t kOffFac = kKQ;
  static constexpr uint32_t kZTile = 64 * 128;                    // do and Z's three terms, two tiles
  static constexpr uint32_t kOffZ = kOffFac + (kFactorBytes + 1023) / 1024 * 1024;
  static constexpr uint32_t kStage = kOffZ + 2 * kZTile;
  // the second image, three terms: one chunk's at a time (there is no room for two at d = 128), loaded when
  // the second product of the chunk before is done with it, a product and three steps before its own
  static constexpr uint32_t kOffImage = kChainStages * kStage;
  static constexpr uint32_t kSTile = kD * 128, kRTile = 128 * 128;
  static constexpr uint32_t kOffS = kOffImage + 3 * kImgTerm;                      // G', three terms
  static constexpr uint32_t kOffR = kOffS + 2 * kSTile;                            // y's and do's rows, three terms
  static constexpr uint32_t kOffBars = kOffR + 2 * kRTile;
  static constexpr uint32_t kSmemBytes = kOffBars + 256 + 1024;
  static constexpr uint32_t kX1 = 0, kX2 = 96, kX3 = 224, kTmem = 512;
  static_assert(kSmemBytes <= 232448, "shared memory above the 227 KB per-block limit");
};
enum : int { kBarY = 4 };   // named barrier of the accumulator warps: y is in shared memory
enum : int { kErrBackLoad = 0x610, kErrBackMma = 0x620, kErrBackAcc = 0x630 };

template <int kD>
__global__ void __launch_bounds__(kChainThreads, 1)
litela_delta_back(const DeltaArgs a, const DeltaGrads gr, const uint8_t* __restrict__ prep, const DeltaSaved saved,
                  int* __restrict__ err) {
  using namespace sm100;
  using Cfg = BackCfg<kD>;
  constexpr int kParts = kD / kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stile = smem + Cfg::kOffS;
  uint8_t* rtile = smem + Cfg::kOffR;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);
  uint64_t* empty = full + kChainStages;
  uint64_t* done = empty + kChainStages;
  uint64_t* s0full = done + 3;
  uint64_t* imgfull = s0full + 1;
  uint64_t* drained = imgfull + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x % kParts, h = (blockIdx.x / kParts) % a.Hv, s = blockIdx.x / (kParts * a.Hv);
  const int hk = h / (a.Hv / a.Hk);
  const DeltaSeq sq = delta_seq(a, s);
  const int nchunk = (sq.len + kChunk - 1) / kChunk;
  const long long slot0 = delta_slot0(a, s, sq);
  const uint8_t* blocks = prep + (slot0 * a.Hv + h) * (long long)kPrepSaveBytes + kPrepFactors;
  const long long block_step = (long long)a.Hv * kPrepSaveBytes;
  constexpr uint32_t kBlock = kFactorBytes + 3 * kImgTerm;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kChainStages; ++i) {
      mbar_init(&full[i], kLoadWarps + 1);
      mbar_init(&empty[i], kAccWarps + 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&done[i], 1);
    mbar_init(s0full, 1);
    mbar_init(imgfull, 1);
    mbar_init(drained, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_holder, Cfg::kTmem);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;

  if (warp < kAccWarps) {
    const int quad = warp & 3, c0 = (warp >> 2) * kN, row = quad * 32 + lane;
    const uint32_t ta = tmem + ((uint32_t)(quad * 32) << 16), tq = ta + (16u << 16);
    const bool has_state = row < kD;
    const int tok = quad * 16 + (lane >> 2), fc = c0 + (lane & 3) * 2;   // chain_frag: tokens tok and tok + 8
    const long long sbase = ((long long)s * a.Hv + h) * (kD * kD) + (long long)row * kD + part * kCols + c0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase, int code) {
      if (ok) ok = mbar_wait(bar, phase & 1, abort_flag, err, kErrBackAcc | code);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after_sync();
    };
    auto hand = [&](int id) {
      fence_proxy_async_smem();
      tc_fence_before_sync();
      bar_arrive(id, kBarThreads);
    };
    F2 S[kN / 2];
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) S[i] = f2(0.f, 0.f);
    if (has_state && gr.dstate_out != nullptr)
#pragma unroll
      for (int i = 0; i < kN; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(gr.dstate_out + sbase + i);
        S[i / 2] = f2(x.x, x.y), S[i / 2 + 1] = f2(x.z, x.w);
      }
    if (nchunk > 0) {
      if (has_state) chain_put<3>(stile, Cfg::kSTile, row, c0, S);
      hand(kBarS);
    }
    for (int it = 0; it < nchunk; ++it) {
      const int n = nchunk - 1 - it, st = it % kChainStages;
      uint8_t* stage = smem + st * Cfg::kStage;
      const long long sh = (slot0 + n) * a.Hv + h;
      wait(&full[st], it / kChainStages, 0);
      const float* fac = reinterpret_cast<const float*>(stage + Cfg::kOffFac);
      float decay[2], to_end[2], beta[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        decay[i] = fac[kFacDecay + tok + 8 * i];
        to_end[i] = fac[kFacToEnd + tok + 8 * i];
        beta[i] = fac[kFacBeta + tok + 8 * i];
      }
      const float chunk_decay = fac[kFacChunk];
      uint32_t dov[kN / 4];
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const int r = tok + (i & 1) * 8, c = fc + (i >> 1) * 8;
        dov[i] = *reinterpret_cast<const uint32_t*>(stage + Cfg::kOffZ + sw128(r, c));
      }
      F2 x[kN / 2], y[kN / 4], z[kN / 4];
      wait(&done[0], it, 1);
      chain_frag<3>(ta + Cfg::kX1, c0, z);
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const float f = to_end[i & 1], mb = -beta[i & 1];
        z[i] = f2_mul(f2(f, f), z[i]);
        x[i] = f2_mul(f2(mb, mb), z[i]);
      }
      chain_put_frag<3, 1>(stage + Cfg::kOffZ, Cfg::kZTile, tok, fc, x);
      hand(kBarR);   // (x, which is -beta Z, goes into the rows' shares too)
      // while the second product runs: do's rows of the third, W
      const float* wp = saved.w + (sh * kChunk + tok) * kD + part * kCols + fc;
      float2 wv[kN / 4];
#pragma unroll
      for (int i = 0; i < kN / 4; ++i)
        wv[i] = __ldg(reinterpret_cast<const float2*>(wp + (i & 1) * 8 * kD + (i >> 1) * 8));
      F2 bdot[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        bdot[i & 1] = f2_fma(x[i], f2(wv[i].x, wv[i].y), bdot[i & 1]);
        const float f = a.scale * decay[i & 1];   // scale e^G do
        x[i] = f2_mul(f2(f, f), f2_bf16(dov[i]));
      }
      chain_put_frag<3>(rtile, Cfg::kRTile, lane_of(tok) + 16, fc, x);
      wait(&done[1], it, 2);
      chain_frag<3>(ta + Cfg::kX2 + 32, c0, x);
      chain_frag<1>(tq + Cfg::kX2, c0, y);
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) {
        const float b = beta[i & 1], md = -decay[i & 1];
        z[i] = f2_add(z[i], f2_add(x[i], y[i]));   // w
        y[i] = f2_mul(f2(b, b), z[i]);
        x[i] = f2_mul(f2(md, md), y[i]);
      }
      chain_put_frag<3>(rtile, Cfg::kRTile, lane_of(tok), fc, x);
      hand(kBarU);
      // while the third product runs: y through Z's second tile to memory, and dv by rows
      float* ytile = reinterpret_cast<float*>(stage + Cfg::kOffZ + Cfg::kZTile);
#pragma unroll
      for (int i = 0; i < kN / 4; ++i)
        *reinterpret_cast<float2*>(ytile + y_off(tok + (i & 1) * 8, fc + (i >> 1) * 8)) = f2_out(y[i]);
      fence_proxy_async_smem();
      bar_sync(kBarY, kAccWarps * 32);
      if (threadIdx.x == 0) {
        bulk_store(gr.y + (sh * kParts + part) * (long long)(Cfg::kZTile / 4), ytile, Cfg::kZTile);
        bulk_commit_group();
      }
      {
        const int r = threadIdx.x >> 2, c = (threadIdx.x & 3) * 8;
        const float4 lo = *reinterpret_cast<const float4*>(ytile + y_off(r, c));
        const float4 hi = *reinterpret_cast<const float4*>(ytile + y_off(r, c + 4));
        if (n * kChunk + r < sq.len)
          *reinterpret_cast<uint4*>(const_cast<__nv_bfloat16*>(delta_row(gr.dv, sq, n * kChunk + r, h)) + part * kCols + c) =
              make_uint4(pack_bf16(lo.x, lo.y), pack_bf16(lo.z, lo.w), pack_bf16(hi.x, hi.y), pack_bf16(hi.z, hi.w));
      }
      F2 sdot = f2(0.f, 0.f);
      wait(s0full, it, 4);   // the state before this chunk, in the tile's place
      if (has_state)
#pragma unroll
        for (int i = 0; i < kN / 8; ++i) {
          const uint4 hi = *reinterpret_cast<const uint4*>(stile + sw128(row, c0 + 8 * i));
          const uint4 lo = *reinterpret_cast<const uint4*>(stile + sw128(row, 32 + c0 + 8 * i));
          const uint4 third = *reinterpret_cast<const uint4*>(stile + Cfg::kSTile + sw128(row, c0 + 8 * i));
          const uint32_t h4[4] = {hi.x, hi.y, hi.z, hi.w}, l4[4] = {lo.x, lo.y, lo.z, lo.w};
          const uint32_t t4[4] = {third.x, third.y, third.z, third.w};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sdot = f2_fma(S[4 * i + q], f2_add(f2_bf16(h4[q]), f2_add(f2_bf16(l4[q]), f2_bf16(t4[q]))), sdot);
        }
      wait(&done[2], it, 3);
      if (has_state) {
        chain_acc<3>(ta + Cfg::kX3, c0, x);
        const F2 d2 = f2(chunk_decay, chunk_decay);
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) S[i] = f2_fma(d2, S[i], x[i]);
        if (n > 0) chain_put<3>(stile, Cfg::kSTile, row, c0, S);
      }
      if (n > 0) hand(kBarS);
      // while the next chunk's first product runs: the rows' shares
      F2 wdot[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < kN / 4; ++i) wdot[i & 1] = f2_fma(z[i], f2(wv[i].x, wv[i].y), wdot[i & 1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 w2 = f2_out(wdot[i]);
        const float2 b2 = f2_out(bdot[i]);
        float wd = w2.x + w2.y, bd = -(b2.x + b2.y);
        wd += __shfl_xor_sync(0xffffffffu, wd, 1);
        bd += __shfl_xor_sync(0xffffffffu, bd, 1);
        wd += __shfl_xor_sync(0xffffffffu, wd, 2);
        bd += __shfl_xor_sync(0xffffffffu, bd, 2);
        float* rw = gr.rows + ((sh * kParts + part) * 4 + (warp >> 2)) * kChunk + tok + 8 * i;
        if ((lane & 3) == 0) {
          rw[0] = wd;
          rw[2 * kChunk] = bd;
        }
      }
      {   // this warp's share of <S0, G'>
        const float2 dd = f2_out(sdot);
        const float dot = sum_warp(dd.x + dd.y);
        if (lane == 0) gr.ends[(sh * kParts + part) * 8 + warp] = dot;
      }
      __syncwarp();
      if (lane == 0) {   // the stage has been read
        if (warp == 0) bulk_wait_group_read<0>();
        mbar_arrive(&empty[st]);
      }
    }
    if (ok && has_state && gr.dstate_in != nullptr)
#pragma unroll
      for (int i = 0; i < kN; i += 4)
        *reinterpret_cast<float4*>(gr.dstate_in + sbase + i) =
            make_float4(f2_out(S[i / 2]).x, f2_out(S[i / 2]).y, f2_out(S[i / 2 + 1]).x, f2_out(S[i / 2 + 1]).y);
  } else if (warp == kIssueWarp) {
    constexpr uint32_t idesc_1 = idesc_bf16_f32(128, 96, false, true);    // [K; Q] G'
    constexpr uint32_t idesc_z = idesc_bf16_f32(128, 128, true, true);    // [X; P T]^T [do, three terms of Z]
    constexpr uint32_t idesc_3 = idesc_bf16_f32(128, 96, true, true);     // .. of the second terms, [do, two of Z]; [K; Q]^T ..
    constexpr uint32_t idesc_2 = idesc_bf16_f32(128, 64, true, true);     // .. of the third terms, [do, one of Z]
    const Desc sdesc = desc_halves(smem_u32(stile), Cfg::kSTile, 1024, kSwizzle128B);
    const Desc rdesc = desc_halves(smem_u32(rtile), Cfg::kRTile, 1024, kSwizzle128B);
    const Desc kqdesc = desc_halves(smem_u32(smem), 16, 1024, kSwizzle128B);
    const Desc imgdesc = desc_halves(smem_u32(smem) + Cfg::kOffImage, kImgBlock, 1024, kSwizzle128B);
    const Desc zdesc = desc_halves(smem_u32(smem) + Cfg::kOffZ, Cfg::kZTile, 1024, kSwizzle128B);
    // [K; Q]^T: M over channels, 128 rows.  d <= 64: rows 64 on of the product take whatever follows
    const Desc ktdesc = desc_halves(smem_u32(smem), kD > 64 ? 16384 : 1024, 1024, kSwizzle128B);
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase, int code) {
      if (ok && lane == 0) ok = mbar_spin(bar, phase & 1, abort_flag, err, kErrBackMma | code);
      ok = __all_sync(0xffffffffu, ok);
    };
    int images = 0;   // loads of an image (lane 0)
    auto load_image = [&](int n) {
      mbar_arrive_expect_tx(imgfull, 3 * kImgTerm);
      bulk_load(smem + Cfg::kOffImage, blocks + n * block_step + kFactorBytes, 3 * kImgTerm, imgfull);
      ++images;
    };
    if (nchunk > 0) {
      if (lane == 0) load_image(nchunk - 1);
      wait(&full[0], 0, 0);
    }
    for (int it = 0; it < nchunk; ++it) {
      const int n = nchunk - 1 - it, st = it % kChainStages;
      const uint32_t off = st * (Cfg::kStage / 16);
      bar_sync(kBarS, kBarThreads);
      tc_fence_after_sync();
      if (lane == 0) {
        bulk_store(gr.gstates + (((slot0 + n) * a.Hv + h) * kParts + part) * (long long)Cfg::kSTile, stile, Cfg::kSTile);
        bulk_commit_group();
        if (ok) {
#pragma unroll
          for (int ks = 0; ks < kD / 16; ++ks)
            umma(tmem + Cfg::kX1, kqdesc + off + (ks / 4) * 1024 + (ks % 4) * 2, sdesc + ks * 128, idesc_1, ks > 0);
          umma_commit(&done[0]);
        }
      }
      __syncwarp();
      wait(imgfull, it, 3);
      bar_sync(kBarR, kBarThreads);
      tc_fence_after_sync();
      if (ok && lane == 0) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma(tmem + Cfg::kX2, imgdesc + ks * 128, zdesc + off + ks * 128, idesc_z, ks > 0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma(tmem + Cfg::kX2, imgdesc + kImgTerm / 16 + ks * 128, zdesc + off + ks * 128, idesc_3, 1u);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          umma(tmem + Cfg::kX2, imgdesc + 2 * kImgTerm / 16 + ks * 128, zdesc + off + ks * 128, idesc_2, 1u);
        umma_commit(&done[1]);
      }
      if (lane == 0) {
        // G' has been read by the first product and stored: the state before the chunk takes its place
        bulk_wait_group_read<0>();
        if (it > 0) mbar_drain(s0full, (it - 1) & 1);   // (long done, unless the walk was given up)
        mbar_arrive_expect_tx(s0full, 2 * Cfg::kSTile);
        bulk_load(stile, saved.states + (((slot0 + n) * a.Hv + h) * kParts + part) * (2LL * Cfg::kSTile), 2 * Cfg::kSTile,
                  s0full);
      }
      __syncwarp();
      bar_sync(kBarU, kBarThreads);
      tc_fence_after_sync();
      if (lane == 0) {
        if (ok) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            umma(tmem + Cfg::kX3, ktdesc + off + ks * 128, rdesc + ks * 128, idesc_3, ks > 0);
          umma_commit(&done[2]);
          umma_commit(&empty[st]);
          // (the accumulator warps have the second product's results: it has read the image)
          if (n > 0) load_image(n - 1);
        }
      }
      __syncwarp();
      if (it + 1 < nchunk) wait(&full[(it + 1) % kChainStages], (it + 1) / kChainStages, 0);
    }
    if (lane == 0) {
      umma_commit(drained);
      mbar_drain(drained, 0);
      bulk_wait_group<0>();
      if (nchunk > 0) {
        mbar_drain(s0full, (nchunk - 1) & 1);
        mbar_drain(imgfull, (images - 1) & 1);
      }
    }
  } else {
    const int t = threadIdx.x - (warp > kIssueWarp ? kAccWarps + 1 : kAccWarps) * 32;
    int issued = 0;
    constexpr int kC = kD / 8, kStep = kLoadThreads / kC, kVC = kCols / 8, kVStep = kLoadThreads / kVC;
    const int r0 = t / kC, c = t % kC, vr0 = t / kVC, vc = t % kVC;
    const uint32_t kq0 = smem_u32(smem) + (c / 8) * 16384 + sw128(lane_of(r0), (c % 8) * 8);
    const uint32_t do0 = smem_u32(smem) + Cfg::kOffZ;
    const long long kstep = kStep * a.k.st, qstep = kStep * a.q.st, dstep = kVStep * gr.dout.st;
    for (int it = 0; it < nchunk; ++it) {
      const int n = nchunk - 1 - it, st = it % kChainStages;
      const bool ok = it < kChainStages || lane != 0 ||
                      mbar_wait(&empty[st], (it / kChainStages - 1) & 1, abort_flag, err, kErrBackLoad | st);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (t == 0) {
        mbar_arrive_expect_tx(&full[st], kFactorBytes);
        bulk_load(smem + st * Cfg::kStage + Cfg::kOffFac, blocks + n * block_step, kFactorBytes, &full[st]);
      }
      issued = it + 1;
      const int n0 = n * kChunk, len = min(kChunk, sq.len - n0);
      const uint32_t dkq = kq0 + st * Cfg::kStage, ddo = do0 + st * Cfg::kStage;
      const __nv_bfloat16* kp = delta_row(a.k, sq, n0 + r0, hk) + c * 8;
      const __nv_bfloat16* qp = delta_row(a.q, sq, n0 + r0, hk) + c * 8;
      const __nv_bfloat16* dp = delta_row(gr.dout, sq, n0 + vr0, h) + part * kCols + vc * 8;
#pragma unroll
      for (int i = 0; i < kChunk / kStep; ++i) {
        const uint32_t o = (dkq ^ (((i * kStep) & 7) << 4)) + lane_of(i * kStep) * 128;
        const bool real = r0 + i * kStep < len;
        cp_async_16(o, real ? kp : a.k.p, real);
        cp_async_16(o + 2048, real ? qp : a.q.p, real);
        kp += kstep;
        qp += qstep;
      }
#pragma unroll
      for (int i = 0; i < kChunk / kVStep; ++i) {
        const int r = vr0 + i * kVStep;
        const bool real = r < len;
        cp_async_16(ddo + sw128(r, vc * 8), real ? dp : gr.dout.p, real);
        dp += dstep;
      }
      if (n > 0) {   // the chunk before into L2
        const int r = n0 - kChunk + t;
        const __nv_bfloat16 *k = delta_row(a.k, sq, r, hk), *q = delta_row(a.q, sq, r, hk);
        prefetch_l2(k);
        prefetch_l2(q);
        if (kD > 64) {
          prefetch_l2(k + 64);
          prefetch_l2(q + 64);
        }
        prefetch_l2(delta_row(gr.dout, sq, r, h) + part * kCols);
        if (t == 0) bulk_prefetch_l2(blocks + (n - 1) * block_step, kBlock);
        if (t == 32)
          bulk_prefetch_l2(saved.states + (((slot0 + n - 1) * a.Hv + h) * kParts + part) * (2LL * Cfg::kSTile), 2 * Cfg::kSTile);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
    }
    if (t == 0 && *abort_flag)
      for (int i = issued > kChainStages ? issued - kChainStages : 0; i < issued; ++i)
        mbar_drain(&full[i % kChainStages], (i / kChainStages) & 1);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, Cfg::kTmem);
  }
}

// ---------------------------------------------------------------------------------------
// litela_delta_grads: dq, dk, dg and dbeta of one chunk and key head per CTA, its value heads one
// after another (their shares of dq and dk are summed in registers, in a fixed order).
//
// mma.sync, 16 warps (d = 32: 8): a warp has 16 rows and a quarter (half) of the columns.  States and
// gradients stream through a ring of tiles of 32 columns.  dg is a sum over do, y, U and S0: the last three
// are entered in three bf16 terms (dg is 2 to 5e-7 off against 64 bits, 1 to 6e-6 with two).  The matrices and
// G', of which dq and dk alone are made, are bf16 pairs: 2^-18 beside the 2^-9 of their results' rounding.  2 x
// 2048 tokens of 16 heads of 128 (8 of keys): 184 us (148 with pairs only), bound by the tensor pipe
// (mma.sync) and, one CTA an SM (registers, shared memory), the waits for the tiles and between the steps;
// 512 CTAs on 148 SMs leave a seventh of the time open.
constexpr int kGradLd = 72;   // row of the 64 x 64 matrices, padded

// d[n] += A B[n] for the first kTerms terms of B[n], the smallest first; one term for all n after the other, so
// that no product waits for the one before it
template <int kTiles, int kTerms, int kWords>
__device__ __forceinline__ void mma_row(float (*d)[4], const uint32_t* a, const uint32_t (*b)[kWords]) {
#pragma unroll
  for (int t = kTerms - 1; t >= 0; --t)
#pragma unroll
    for (int n = 0; n < kTiles; ++n) sm100::mma_16816(d[n], a, b[n] + 2 * t);
}

template <int kD>
struct GradCfg {
  static constexpr int kCW = kD >= 64 ? 4 : 2;                     // warps beside one another
  static constexpr int kThreads = 4 * kCW * 32;
  static constexpr int kLd = kD + 8;
  static constexpr uint32_t kRows = kChunk * kLd * 2;              // 64 rows of d, bf16
  static constexpr uint32_t kTile = kD * 128;
  static constexpr uint32_t kOffK = 0, kOffQ = kRows, kOffDo = 2 * kRows;
  static constexpr uint32_t kOffU = 3 * kRows, kOffY = 6 * kRows;  // three terms each
  static constexpr uint32_t kOffM = 9 * kRows;                     // M1 . D and M2 . D, pairs
  static constexpr uint32_t kMat = kChunk * kGradLd * 2;
  static constexpr uint32_t kOffTile = (kOffM + 4 * kMat + 127) / 128 * 128;
  static constexpr int kRing = kD > 64 ? 2 : 3;                    // tiles of states in shared memory
  // S0's third terms, a tile of 64-byte rows for each 32 columns; at d = 128 in the matrices' place, after them
  static constexpr uint32_t kThirdTile = kD * 64;
  static constexpr bool kThirdLate = kD > 64;
  static constexpr uint32_t kOffThird = kThirdLate ? kOffM : kOffTile + kRing * kTile;
  static_assert(!kThirdLate || kD / 32 * kThirdTile <= 4 * kMat, "third terms");
  static constexpr uint32_t kOffFac = kThirdLate ? kOffTile + kRing * kTile : kOffThird + kD / 32 * kThirdTile;   // the prepared block's factors
  // sums of dg: by token for the warps beside one another, N's columns for the 4 below
  static constexpr uint32_t kOffSum = kOffFac + kFactorBytes;
  static constexpr uint32_t kSmemBytes = kOffSum + (kCW + 4) * kChunk * 4 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory above the 227 KB per-block limit");
};

template <int kD>
__global__ void __launch_bounds__(GradCfg<kD>::kThreads, 1)
litela_delta_grads(const DeltaArgs a, const DeltaGrads gr, const uint8_t* __restrict__ prep, const DeltaSaved saved) {
  using namespace sm100;
  using Cfg = GradCfg<kD>;
  constexpr int kThreads = Cfg::kThreads, kCW = Cfg::kCW;
  constexpr int kParts = kD / 32, kT = kD / 8 / kCW;   // kT: tiles of 8 columns of d that a warp has
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* fac = reinterpret_cast<float*>(smem + Cfg::kOffFac);
  const float *rowf = fac + kFacRow, *colf = fac + kFacCol;
  const float2* rel = reinterpret_cast<const float2*>(fac + kFacRel);
  float* rsum = reinterpret_cast<float*>(smem + Cfg::kOffSum);
  float* csum = rsum + kCW * kChunk;

  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g4 = lane >> 2, t2 = (lane & 3) * 2;
  const int rb = w / kCW, cw = w % kCW, l8 = lane & 7, k8 = ((lane >> 3) & 1) * 8;
  const int slot = blockIdx.x / a.Hk, hk = blockIdx.x - slot * a.Hk, group = a.Hv / a.Hk;
  if (a.zero_rest) {
    delta_zero_rest(a, gr.dq, a.Hk, kD);
    delta_zero_rest(a, gr.dk, a.Hk, kD);
    delta_zero_rest(a, gr.dv, a.Hv, kD);
    delta_rest(a, a.Hv, [&](int row, int h) { gr.dg[(long long)row * a.Hv + h] = gr.dbeta[(long long)row * a.Hv + h] = 0.f; });
  }
  int s, n0;
  DeltaSeq sq;
  if (!delta_find(a, slot, lane, s, sq, n0)) {
    pdl_wait_primary();   // (a grid that is all such blocks may not end before litela_delta_back)
    return;
  }
  const int len = min(kChunk, sq.len - n0);
  const uint32_t base = smem_u32(smem);

  // 64 rows of a view into shared memory
  auto copy_rows = [&](const DeltaView& v, int head, uint32_t dst) {
    constexpr int kC = kD / 8, kStep = kThreads / kC;
    const int c = tid % kC, r0 = tid / kC;
    const __nv_bfloat16* p = delta_row(v, sq, n0 + r0, head) + c * 8;
#pragma unroll
    for (int i = 0; i < kChunk / kStep; ++i) {
      const bool real = r0 + i * kStep < len;
      cp_async_16(base + dst + (r0 + i * kStep) * (Cfg::kLd * 2) + c * 16, real ? p : v.p, real);
      p += kStep * v.st;
    }
  };
  copy_rows(a.k, hk, Cfg::kOffK);
  copy_rows(a.q, hk, Cfg::kOffQ);
  pdl_wait_primary();   // y, G' and the shares come from litela_delta_back

  float dq[kT][4], dk[kT][4];
#pragma unroll
  for (int n = 0; n < kT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) dq[n][i] = dk[n][i] = 0.f;

#pragma unroll 1
  for (int hv = 0; hv < group; ++hv) {
    const int h = hk * group + hv;
    const long long sh = (long long)slot * a.Hv + h;
    // tile p of the states (p < kParts), then of the gradients
    auto load_tile = [&](int p) {
      const uint8_t* src = (p < kParts ? saved.states + (sh * kParts + p) * (2LL * Cfg::kTile)   // the first two terms
                                       : gr.gstates + (sh * kParts + p - kParts) * (long long)Cfg::kTile);
      const uint32_t dst = base + Cfg::kOffTile + (p % Cfg::kRing) * Cfg::kTile;
#pragma unroll 1
      for (int i = tid * 16; i < (int)Cfg::kTile; i += kThreads * 16) cp_async_16(dst + i, src + i, true);
    };
    copy_rows(gr.dout, h, Cfg::kOffDo);
    if (tid < (int)kFactorBytes / 16) cp_async_16(base + Cfg::kOffFac + tid * 16, prep + sh * kPrepSaveBytes + kPrepFactors + tid * 16, true);
    auto load_thirds = [&] {   // rows of 4 pieces of 16 bytes, from S0's second tiles; row pairs share 128 bytes
#pragma unroll 1
      for (int i = tid; i < kParts * kD * 4; i += kThreads) {
        const int p = i / (kD * 4), r = (i >> 2) % kD, c = i & 3;
        cp_async_16(base + Cfg::kOffThird + p * Cfg::kThirdTile + r * 64 + ((c ^ (r >> 1)) & 3) * 16,
                    saved.states + ((sh * kParts + p) * 2 + 1) * (long long)Cfg::kTile + sw128(r, c * 8), true);
      }
    };
    if (!Cfg::kThirdLate) load_thirds();
#pragma unroll
    for (int p = 0; p < Cfg::kRing - 1; ++p) {
      load_tile(p);
      cp_async_commit();
    }
    // this token's w . W and b (tid < 64); W's values: all in flight at once
    constexpr int kQ = kChunk * kD / 4 / kThreads;   // 4 columns of a row at a time
    float4 wv[kQ];
    const float4* wp = reinterpret_cast<const float4*>(saved.w + sh * kChunk * kD) + tid;
#pragma unroll
    for (int i = 0; i < kQ; ++i) wv[i] = __ldg(wp + i * kThreads);
    float4 yv[kQ];
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const int q = i * kThreads + tid, r = q / (kD / 4), c = (q % (kD / 4)) * 4;
      yv[i] = __ldcg(reinterpret_cast<const float4*>(gr.y + (sh * kParts + c / 32) * (kChunk * 32) + y_off(r, c % 32)));
    }
    float wd = 0.f, bd = 0.f, end = 0.f;
    if (tid < kChunk) {
      const float* rw = gr.rows + sh * kParts * 4 * kChunk + tid;   // [part][which][half][token]
      float x[kParts][4];
#pragma unroll
      for (int p = 0; p < kParts; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[p][i] = __ldcg(rw + (p * 4 + i) * kChunk);
      if (lane < kParts * 8) end = __ldcg(gr.ends + sh * kParts * 8 + lane);
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        wd += x[p][0] + x[p][1];
        bd += x[p][2] + x[p][3];
      }
      end = sum_warp(end);
    }
    cp_async_wait<Cfg::kRing - 2>();   // do, the factors and the first tile (K and Q)
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQ; ++i) {   // U = beta W, and y
      const int q = i * kThreads + tid, r = q / (kD / 4), c = (q % (kD / 4)) * 4;
      const float f = fac[kFacBeta + r];
      uint32_t u[3][2], y[3][2];
      split_terms(f * wv[i].x, f * wv[i].y, &u[0][0], 2);
      split_terms(f * wv[i].z, f * wv[i].w, &u[0][1], 2);
      split_terms(yv[i].x, yv[i].y, &y[0][0], 2);
      split_terms(yv[i].z, yv[i].w, &y[0][1], 2);
      uint8_t* dst = smem + Cfg::kOffU + (r * Cfg::kLd + c) * 2;
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        *reinterpret_cast<uint2*>(dst + t * Cfg::kRows) = make_uint2(u[t][0], u[t][1]);
        *reinterpret_cast<uint2*>(dst + Cfg::kOffY - Cfg::kOffU + t * Cfg::kRows) = make_uint2(y[t][0], y[t][1]);
      }
    }
    __syncthreads();

    // M1 = do U^T, M2 = y U^T, Q K^T and K K^T: rows 16 rb .., of the 2 rb + 2 tiles of columns up to the diagonal block
    // cw, cw + kCW, ..  (d: K dimension; tiles beyond are computed along and not kept)
    constexpr int kMT = 8 / kCW;
    float sums[2];   // this thread's share of the tokens' sums, rows r0 and r0 + 8
    {
      float m1[kMT][4], m2[kMT][4], qk[kMT][4], kk[kMT][4];
#pragma unroll
      for (int n = 0; n < kMT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) m1[n][i] = m2[n][i] = qk[n][i] = kk[n][i] = 0.f;
      const uint32_t arow = (16 * rb + (lane & 15)) * (Cfg::kLd * 2) + (lane >> 4) * 16;
      // matrices by lane / 8: first term of 0..7 and 8..15 of the K dimension, second; third of two tiles of columns
      const uint32_t brow = base + Cfg::kOffU + (lane >> 4) * Cfg::kRows + (8 * cw + l8) * (Cfg::kLd * 2) + k8 * 2;
      const uint32_t trow = base + Cfg::kOffU + 2 * Cfg::kRows + (8 * (cw + (lane >> 4) * kCW) + l8) * (Cfg::kLd * 2) + k8 * 2;
      // K's: two tiles of columns
      const uint32_t krow = base + Cfg::kOffK + (8 * (cw + (lane >> 4) * kCW) + l8) * (Cfg::kLd * 2) + k8 * 2;
#pragma unroll 1
      for (int ks = 0; ks < kD / 16; ++ks) {
        uint32_t ad[4], ya[3][4];
        {
          uint32_t aq[4], ak[4];
          ldmatrix_x4(aq, base + Cfg::kOffQ + arow + ks * 32);
          ldmatrix_x4(ak, base + Cfg::kOffK + arow + ks * 32);
#pragma unroll
          for (int n = 0; n < kMT; n += 2) {
            uint32_t b[4];
            ldmatrix_x4(b, krow + n * 8 * kCW * (Cfg::kLd * 2) + ks * 32);
#pragma unroll
            for (int e = 0; e < 2; ++e) mma_16816(qk[n + e], aq, b + 2 * e);
#pragma unroll
            for (int e = 0; e < 2; ++e) mma_16816(kk[n + e], ak, b + 2 * e);
          }
        }
        ldmatrix_x4(ad, base + Cfg::kOffDo + arow + ks * 32);
#pragma unroll
        for (int t = 0; t < 3; ++t) ldmatrix_x4(ya[t], base + Cfg::kOffY + t * Cfg::kRows + arow + ks * 32);
        uint32_t b[kMT][6];   // terms of 8 columns
#pragma unroll
        for (int n = 0; n < kMT; n += 2) {
          uint32_t third[4];
          ldmatrix_x4(third, trow + n * 8 * kCW * (Cfg::kLd * 2) + ks * 32);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ldmatrix_x4(b[n + e], brow + (n + e) * 8 * kCW * (Cfg::kLd * 2) + ks * 32);
            b[n + e][4] = third[2 * e], b[n + e][5] = third[2 * e + 1];
          }
        }
        mma_row<kMT, 3, 6>(m1, ad, b);
        mma_row<kMT, 1, 6>(m2, ya[2], b);
        mma_row<kMT, 2, 6>(m2, ya[1], b);
        mma_row<kMT, 3, 6>(m2, ya[0], b);
      }
      // by D; M1 by scale, M2 negated; N's sums of the warp's rows and columns
      float nrow[2] = {0.f, 0.f};
#pragma unroll
      for (int n = 0; n < kMT; ++n) {
        float ncol[2] = {0.f, 0.f};
        if (cw + kCW * n < 2 * rb + 2) {
          const int c = 8 * (cw + kCW * n) + t2;
          const bool diag = c >= 16 * rb;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int r = 16 * rb + g4 + 8 * q;
            float d[2];
            if (diag) {
              const float2 rr = rel[r], ra = rel[c], rc = rel[c + 1];
              d[0] = expf((rr.x - ra.x) + (rr.y - ra.y));
              d[1] = expf((rr.x - rc.x) + (rr.y - rc.y));
            } else {
              const float2 cf = *reinterpret_cast<const float2*>(colf + rb * 48 + c);
              d[0] = rowf[r] * cf.x, d[1] = rowf[r] * cf.y;
            }
            uint32_t hi, lo;
            uint8_t* dst = smem + Cfg::kOffM + (r * kGradLd + c) * 2;
            const float p0 = c <= r ? a.scale * d[0] * m1[n][2 * q] : 0.f, p1 = c + 1 <= r ? a.scale * d[1] * m1[n][2 * q + 1] : 0.f;
            const float l0 = c < r ? -d[0] * m2[n][2 * q] : 0.f, l1 = c + 1 < r ? -d[1] * m2[n][2 * q + 1] : 0.f;
            const float n0 = c < r ? p0 * qk[n][2 * q] + l0 * kk[n][2 * q] : 0.f;
            const float n1 = c + 1 < r ? p1 * qk[n][2 * q + 1] + l1 * kk[n][2 * q + 1] : 0.f;
            nrow[q] += n0 + n1;
            ncol[0] += n0, ncol[1] += n1;
            split_bf16(p0, p1, hi, lo);
            *reinterpret_cast<uint32_t*>(dst) = hi;
            *reinterpret_cast<uint32_t*>(dst + Cfg::kMat) = lo;
            split_bf16(l0, l1, hi, lo);
            *reinterpret_cast<uint32_t*>(dst + 2 * Cfg::kMat) = hi;
            *reinterpret_cast<uint32_t*>(dst + 3 * Cfg::kMat) = lo;
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) ncol[e] += __shfl_xor_sync(0xffffffffu, ncol[e], o);
          if (lane < 4) csum[rb * kChunk + 8 * (cw + kCW * n) + t2 + e] = ncol[e];
        }
      }
      sums[0] = nrow[0], sums[1] = nrow[1];
    }
    __syncthreads();

    // the 64 x 64 matrices with K and Q: the warp's columns of dq and dk
    {
      const uint32_t kcol = base + Cfg::kOffK + (l8 + k8) * (Cfg::kLd * 2) + cw * (kT * 16) + (lane >> 4) * 16;   // two tiles
      const uint32_t qcol = kcol + (Cfg::kOffQ - Cfg::kOffK);
      const uint32_t mrow = base + Cfg::kOffM + ((16 * rb + (lane & 15)) * kGradLd + (lane >> 4) * 8) * 2;
#pragma unroll 1
      for (int kb = 0; kb <= rb; ++kb) {   // rows 16 rb: blocks up to the diagonal
        uint32_t ah[4], al[4], ch[4], cl[4];
        ldmatrix_x4(ah, mrow + kb * 32);
        ldmatrix_x4(al, mrow + Cfg::kMat + kb * 32);
        ldmatrix_x4(ch, mrow + 2 * Cfg::kMat + kb * 32);
        ldmatrix_x4(cl, mrow + 3 * Cfg::kMat + kb * 32);
#pragma unroll
        for (int n = 0; n < kT; n += 2) {
          uint32_t b[4];   // tile n: b[0], b[1]; tile n + 1: b[2], b[3]
          ldmatrix_x4_t(b, kcol + kb * 16 * (Cfg::kLd * 2) + n * 16);
#pragma unroll
          for (int e = 0; e < 2; ++e) mma_16816(dq[n + e], al, b + 2 * e);
#pragma unroll
          for (int e = 0; e < 2; ++e) mma_16816(dk[n + e], cl, b + 2 * e);
#pragma unroll
          for (int e = 0; e < 2; ++e) mma_16816(dq[n + e], ah, b + 2 * e);
#pragma unroll
          for (int e = 0; e < 2; ++e) mma_16816(dk[n + e], ch, b + 2 * e);
        }
      }
      // transposed: rows of dk are columns of the matrices
      const uint32_t mcol = base + Cfg::kOffM + ((l8 + (lane >> 4) * 8) * kGradLd + 16 * rb + k8) * 2;
#pragma unroll 1
      for (int kb = rb; kb < 4; ++kb) {
        uint32_t ah[4], al[4], ch[4], cl[4];
        const uint32_t o = mcol + kb * 16 * kGradLd * 2;
        ldmatrix_x4_t(ah, o);
        ldmatrix_x4_t(al, o + Cfg::kMat);
        ldmatrix_x4_t(ch, o + 2 * Cfg::kMat);
        ldmatrix_x4_t(cl, o + 3 * Cfg::kMat);
#pragma unroll
        for (int n = 0; n < kT; n += 2) {
          uint32_t b[4], c[4];
          ldmatrix_x4_t(b, qcol + kb * 16 * (Cfg::kLd * 2) + n * 16);
          ldmatrix_x4_t(c, kcol + kb * 16 * (Cfg::kLd * 2) + n * 16);
#pragma unroll
          for (int e = 0; e < 2; ++e) mma_16816(dk[n + e], al, b + 2 * e);
#pragma unroll
          for (int e = 0; e < 2; ++e) mma_16816(dk[n + e], cl, c + 2 * e);
#pragma unroll
          for (int e = 0; e < 2; ++e) mma_16816(dk[n + e], ah, b + 2 * e);
#pragma unroll
          for (int e = 0; e < 2; ++e) mma_16816(dk[n + e], ch, c + 2 * e);
        }
      }
    }
    // do S0^T, y S0^T, then U G'^T, 32 columns of the state (K dimension) at a time
    const int r0 = 16 * rb + g4;
    const uint32_t arow = (16 * rb + (lane & 15)) * (Cfg::kLd * 2) + (lane >> 4) * 16;
    auto tile_b = [&](uint32_t* b, int p, int n, int ks) {   // rows (channels) of the tile: hi, lo
      const int row = (cw * kT + n) * 8 + l8, col = 16 * ks + k8 + (lane >> 4) * 32;
      ldmatrix_x4(b, base + Cfg::kOffTile + (p % Cfg::kRing) * Cfg::kTile + sw128(row, col));
    };
    // the warp's columns of rows r0 and r0 + 8 of x with those of K or Q; and such sums for all warps to add
    auto with_rows = [&](uint32_t off, const float (*x)[4], float* d) {
#pragma unroll
      for (int n = 0; n < kT; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t v = *reinterpret_cast<const uint32_t*>(smem + off + ((r0 + 8 * q) * Cfg::kLd + (cw * kT + n) * 8 + t2) * 2);
          d[q] += x[n][2 * q] * __uint_as_float(v << 16) + x[n][2 * q + 1] * __uint_as_float(v & 0xFFFF0000u);
        }
    };
    auto put_rows = [&](float* dst, float* d) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        d[q] += __shfl_xor_sync(0xffffffffu, d[q], 1);
        d[q] += __shfl_xor_sync(0xffffffffu, d[q], 2);
        if ((lane & 3) == 0) dst[cw * kChunk + r0 + 8 * q] = d[q];
      }
    };
    {
      float x[kT][4], y[kT][4];
#pragma unroll
      for (int n = 0; n < kT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = y[n][i] = 0.f;
#pragma unroll 1
      for (int p = 0; p < kParts; ++p) {
        if (p + Cfg::kRing - 1 < 2 * kParts) load_tile(p + Cfg::kRing - 1);
        cp_async_commit();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          uint32_t ad[4], ya[3][4];
          const uint32_t o = arow + (2 * p + ks) * 32;
          ldmatrix_x4(ad, base + Cfg::kOffDo + o);
#pragma unroll
          for (int t = 0; t < 3; ++t) ldmatrix_x4(ya[t], base + Cfg::kOffY + t * Cfg::kRows + o);
          constexpr int kM = kT < 4 ? kT : 4;
#pragma unroll
          for (int m = 0; m < kT; m += kM) {
            uint32_t b[kM][4];
#pragma unroll
            for (int n = 0; n < kM; ++n) tile_b(b[n], p, m + n, ks);
            mma_row<kM, 2, 4>(x + m, ad, b);
            mma_row<kM, 1, 4>(y + m, ya[2], b);
            mma_row<kM, 2, 4>(y + m, ya[1], b);
            mma_row<kM, 2, 4>(y + m, ya[0], b);
          }
        }
        cp_async_wait<Cfg::kRing - 2>();
        __syncthreads();   // the next tile has landed, and everyone is done with this one's neighbour
        if (Cfg::kThirdLate && p == 0) {   // (and with the matrices)
          load_thirds();
          cp_async_commit();
        }
      }
      // S0's third terms: matrices by lane / 8: 8 of the 32 columns
#pragma unroll 1
      for (int p = 0; p < kParts; ++p) {
        uint32_t ad[2][4], ya[2][4];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          ldmatrix_x4(ad[ks], base + Cfg::kOffDo + arow + (2 * p + ks) * 32);
          ldmatrix_x4(ya[ks], base + Cfg::kOffY + arow + (2 * p + ks) * 32);
        }
#pragma unroll
        for (int n = 0; n < kT; ++n) {
          uint32_t b[4];
          const int row = (cw * kT + n) * 8 + l8;
          ldmatrix_x4(b, base + Cfg::kOffThird + p * Cfg::kThirdTile + row * 64 + (((lane >> 3) ^ (row >> 1)) & 3) * 16);
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            mma_16816(x[n], ad[ks], b + 2 * ks);
            mma_16816(y[n], ya[ks], b + 2 * ks);
          }
        }
      }
      const float e0 = fac[kFacDecay + r0], e1 = fac[kFacDecay + r0 + 8];
#pragma unroll
      for (int n = 0; n < kT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = i < 2 ? e0 : e1;
          x[n][i] *= a.scale * e;
          y[n][i] *= -e;
          dq[n][i] += x[n][i];
          dk[n][i] += y[n][i];
        }
      with_rows(Cfg::kOffQ, x, sums);
      with_rows(Cfg::kOffK, y, sums);
      put_rows(rsum, sums);
    }
    {
      float x[kT][4];
#pragma unroll
      for (int n = 0; n < kT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[n][i] = 0.f;
#pragma unroll 1
      for (int p = kParts; p < 2 * kParts; ++p) {
        if (p + Cfg::kRing - 1 < 2 * kParts) load_tile(p + Cfg::kRing - 1);
        cp_async_commit();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          uint32_t uh[4], ul[4];
          const uint32_t o = arow + (2 * (p - kParts) + ks) * 32;
          ldmatrix_x4(uh, base + Cfg::kOffU + o);
          ldmatrix_x4(ul, base + Cfg::kOffU + Cfg::kRows + o);
          constexpr int kM = kT < 4 ? kT : 4;
#pragma unroll
          for (int m = 0; m < kT; m += kM) {
            uint32_t b[kM][4];
#pragma unroll
            for (int n = 0; n < kM; ++n) tile_b(b[n], p, m + n, ks);
            mma_row<kM, 1, 4>(x + m, ul, b);
            mma_row<kM, 2, 4>(x + m, uh, b);
          }
        }
        cp_async_wait<Cfg::kRing - 2>();
        __syncthreads();
      }
      const float e0 = fac[kFacToEnd + r0], e1 = fac[kFacToEnd + r0 + 8];
#pragma unroll
      for (int n = 0; n < kT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) dk[n][i] += (i < 2 ? e0 : e1) * x[n][i];
    }
    __syncthreads();
    if (tid < kChunk) {
      // the sums over the tokens from this one on and over those before it: inside the warp, then the
      // other warp's; N's columns beyond the rows of a block are zero
      float x = 0.f, b = bd;
#pragma unroll
      for (int i = 0; i < kCW; ++i) x += rsum[i * kChunk + tid];
#pragma unroll
      for (int i = 0; i < 4; ++i) x -= csum[i * kChunk + tid];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float up = __shfl_down_sync(0xffffffffu, x, o), down = __shfl_up_sync(0xffffffffu, b, o);
        if (lane + o < 32) x += up;
        if (lane >= o) b += down;
      }
      float pre = __shfl_up_sync(0xffffffffu, b, 1);   // (not b - bd: that loses small sums beside a large one)
      if (lane == 0) pre = 0.f;
      asm volatile("barrier.cta.sync 1, 64;" ::: "memory");   // (rsum has been read)
      if (tid == 32) rsum[0] = x;
      if (tid == 31) rsum[1] = b;
      asm volatile("barrier.cta.sync 1, 64;" ::: "memory");
      x += pre + (tid < 32 ? rsum[0] : rsum[1]);
      if (tid < len) {
        const long long o = ((long long)sq.entry * a.ntok + sq.first + n0 + tid) * a.Hv + h;
        gr.dbeta[o] = wd;
        gr.dg[o] = x + fac[kFacChunk] * end;
      }
    }
    __syncthreads();
  }

#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int r = 16 * rb + g4 + 8 * q;
    if (r < len) {
      __nv_bfloat16* dqp = const_cast<__nv_bfloat16*>(delta_row(gr.dq, sq, n0 + r, hk)) + cw * kT * 8 + t2;
      __nv_bfloat16* dkp = const_cast<__nv_bfloat16*>(delta_row(gr.dk, sq, n0 + r, hk)) + cw * kT * 8 + t2;
#pragma unroll
      for (int n = 0; n < kT; ++n) {
        *reinterpret_cast<uint32_t*>(dqp + 8 * n) = pack_bf16(dq[n][2 * q], dq[n][2 * q + 1]);
        *reinterpret_cast<uint32_t*>(dkp + 8 * n) = pack_bf16(dk[n][2 * q], dk[n][2 * q + 1]);
      }
    }
  }
}

}  // namespace litela
