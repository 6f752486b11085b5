// The gated delta rule by chunks of 64 steps, backwards: the adjoint of the state from
// chunk to chunk, one block per (sequence, head) (bf16 inputs; records of
// csrc/delta_prep.cu, formulas in delta.cuh).
//
// The mirror of csrc/delta_chunk.cu. For one chunk whose end has the adjoint X:
//   dU^T = (X^T K^T) diag(exp(G_64 - G)) + dY^T A      du = dU through Tb: du^T = dU^T Tb
//   dv = beta du
//   X'^T = exp(G_64) X^T + scale (dY diag(exp G))^T Q - (dv diag(exp G))^T K
// Rows are the value's columns p again; X, dU, dv and dY diag(exp G) are split into three
// bf16 parts on the way to X, dY and the records' parts are exact as they are. The chain is
// K X -> Tb -> K^T dv; dY^T A and Q^T dY run in its pauses.
// Written: dv, du (fp32), X at each chunk's end, dh0.
#pragma once

#include "delta.cuh"
#include "delta_chunk.cuh"
#include "sm100.cuh"

namespace pdssm {
namespace chunk_bwd {

using namespace sm100;

constexpr int kStateWarps = 8, kIssuer = 8, kLoader0 = 9, kLoaders = 2;

// kX, kR, kU: [half], from the four warps that have that half of a row's columns.
enum Bar { kFull, kFree = kFull + 3, kX = kFree + 3, kR = kX + 2, kU = kR + 2, kDoneS = kU + 2, kDoneU, kDoneD, kEnd, kBars };

template <int NP, int PM>
struct Layout {
  // tensor memory: P holds X's parts, then those of dv; D the parts of dU, then the update;
  // Q the parts of dY diag(exp G); Y dY itself; Z first X^T K^T, then du; A dY^T A.
  static constexpr int kP = 0, kPn = 3 * NP / 2, kD = kPn, kDn = NP > 96 ? NP : 96;
  static constexpr int kQ = NP == 128 ? kP + 96 : kD + kDn, kZ = (NP == 128 ? kD : kQ) + (NP == 128 ? kDn : 96);
  static constexpr int kA = kZ + 64, kY = kA + 64, kCols = 512;
  static_assert(kY + 32 <= kCols, "columns");
  static constexpr int kTile = (NP / 8) * kChunkGroup, kDy = kChunk * PM * 2, kRec = 6 * kSquare + kScalars;
  static constexpr int kDyOff = 2 * kTile, kRecOff = kDyOff + kDy, kStage = kRecOff + kRec;
  static constexpr int kStages = 3 * kStage + 256 <= 227 * 1024 ? 3 : 2;  // three where they fit
  static constexpr int kBarOff = kStages * kStage, kBytes = kBarOff + 8 * kBars + 16;
  static constexpr int kParts = 256 / PM, W = kChunk / kParts, WN = NP / kParts;
};

// One sequence of one head, columns p0 ...
template <int NP, int PM>
__device__ __forceinline__ void run(const DeltaArgs &a, bool wide, bool wide_v, int p0) {
  using Lay = Layout<NP, PM>;
  constexpr int W = Lay::W, WN = Lay::WN;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::kBarOff);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + kBars);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int64_t h = blockIdx.y, b = blockIdx.z, bh = b * a.H + h, hk = h / (a.H / a.Hk);
  const int64_t len = live_steps(a.lengths, b, a.L);
  const int chunks = __shfl_sync(0xffffffffu, (int)((len + kChunk - 1) / kChunk), 0);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) {
      const bool half = i >= kX && i < kDoneS, state = i >= kFree && i < kX;
      mbar_init(&bars[i], half ? kStateWarps / 2 : state ? kStateWarps : i < kFree ? 32 * kLoaders + 1 : 1);
    }
    mbar_fence_init();
  }
  if (warp == kIssuer) {
    tmem_alloc(tslot, Lay::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, *tslot, 0);

  // Every wait of a role on another is bounded. When one has run out, anywhere in the launch, all waits that
  // are not over end, and each role leaves its loop at its next unfinished wait, a warp (the loaders) as one:
  // nothing works on operands that are not there. The loaders and the issuer then wait for their own
  // copies and products, and the block ends.
  const auto wait = [&](int which, uint32_t parity) { return __all_sync(0xffffffffu, wait_bar(&bars[which], parity, a.err, a.wait_ns)); };

  // Turn i works on chunk chunks - 1 - i.
  if (warp >= kLoader0 + kLoaders) {
    // the block has one warp more than this needs
  } else if (warp >= kLoader0) {
    const int tid = threadIdx.x - 32 * kLoader0;
    const bool copies = wide && wide_v && a.N == NP && a.P - p0 >= PM;  // nothing is written by the threads themselves
    using B = const __nv_bfloat16;
    const auto go_on = [&](int which, uint32_t parity) {
      return all_of<32 * kLoaders>(wait_bar(&bars[which], parity, a.err, a.wait_ns));
    };
    int issued = 0;
    // a short limit runs out here: nothing has been asked for yet
    if (a.wait_ns < kShortNs && chunks > 0) all_of<32 * kLoaders>(wait_slow<false>(&bars[kFull], 0, a.err, a.wait_ns));
    for (int i = 0, s = 0, turn = 0; i < chunks; ++i) {
      const int chunk = chunks - 1 - i;
      if (turn && !go_on(kFree + s, (turn - 1) & 1)) break;
      uint8_t *st = smem + s * Lay::kStage;
      uint64_t *full = &bars[kFull + s];
      const int live = (int)min((int64_t)kChunk, len - (int64_t)chunk * kChunk);
      const int64_t row0 = b * a.L + (int64_t)chunk * kChunk;
      const bool whole = copies && live == kChunk;
      if (tid < 32) {
        if (lane == 0) {
          mbar_expect_tx(full, Lay::kRec);
          bulk_load(st + Lay::kRecOff, a.records + (bh * a.nC + chunk) * a.rec_bytes + 3 * kSquare, Lay::kRec, full);
        }
      }
      load_tile<NP / 8, kChunkGroup, 16, 32 * kLoaders>(st, static_cast<B *>(a.k), row0, a.Hk, hk, a.N, 0, live, wide, tid);
      load_tile<NP / 8, kChunkGroup, 16, 32 * kLoaders>(st + Lay::kTile, static_cast<B *>(a.q), row0, a.Hk, hk, a.N, 0, live, wide, tid);
      load_tile<PM / 8, 16, 2 * PM, 32 * kLoaders>(st + Lay::kDyOff, static_cast<B *>(a.dy), row0, a.H, h, a.P, p0, live, wide_v, tid);
      if (whole) {
        cp_async_arrive(full);  // on to the next chunk while the copies land
      } else {
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(full);
      }
      if (++s == Lay::kStages) s = 0, ++turn;
      ++issued;
    }
    for (int i = max(issued - Lay::kStages, 0); i < issued; ++i) wait_own(&bars[kFull + i % Lay::kStages], (i / Lay::kStages) & 1, a.err);
  } else if (warp == kIssuer) {
    constexpr uint32_t idS = idesc_bf16_f32(PM, kChunk, false, false), idT = idesc_bf16_f32(PM, kChunk, false, true),
                       idD = idesc_bf16_f32(PM, NP, false, true);
    const uint32_t base = smem_u32(smem);
    for (int i = 0, s = 0, turn = 0; i < chunks; ++i) {
      const uint32_t ph = i & 1, sk = base + s * Lay::kStage, sq = sk + Lay::kTile, tb = sk + Lay::kRecOff, sa = tb + 3 * kSquare;
      const uint64_t dk = smem_desc(sk, kChunkGroup, 128), dkt = smem_desc(sk, 128, kChunkGroup), dqt = smem_desc(sq, 128, kChunkGroup),
                     dtb = smem_desc(tb, 128, 1024), da = smem_desc(sa, 128, 1024);
      if (!wait(kFull + s, turn & 1)) goto issued_all;
      fence_proxy_async_smem();  // the loaders' writes, seen through the barrier, before the tensor core's reads
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        if (!wait(kX + f, ph)) goto issued_all;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int q = 2; q >= 0; --q)
#pragma unroll
            for (int ks = f * NP / 32; ks < (f + 1) * NP / 32; ++ks)
              mma_bf16_ts(tbase + Lay::kZ, tbase + Lay::kP + q * (NP / 2) + 8 * ks, dk + (2 * kChunkGroup * ks >> 4), idS, f + (2 - q) + ks > 0);
          if (f == 1) {
#pragma unroll
            for (int q = 2; q >= 0; --q)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_bf16_ts(tbase + Lay::kA, tbase + Lay::kY + 8 * ks, da + ((q * kSquare + 256 * ks) >> 4), idT, (2 - q) + ks > 0);
            mma_commit(&bars[kDoneS]);
          }
        }
        __syncwarp();
      }
      // du takes the place of X^T K^T, so all warps have to have read that
      if (!wait(kR, ph)) goto issued_all;
      if (!wait(kR + 1, ph)) goto issued_all;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int o = 2; o >= 0; --o)
#pragma unroll
          for (int q = 0; q <= o; ++q)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_bf16_ts(tbase + Lay::kZ, tbase + Lay::kD + (o - q) * 32 + 8 * ks, dtb + ((q * kSquare + 256 * ks) >> 4), idT,
                          (2 - o) + q + ks > 0);
        mma_commit(&bars[kDoneU]);
      }
      __syncwarp();
      // kU also says that the half's parts of dY diag(exp G) are there
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        if (!wait(kU + f, ph)) goto issued_all;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int q = 2; q >= 0; --q)
#pragma unroll
            for (int ks = 2 * f; ks < 2 * f + 2; ++ks) {
              mma_bf16_ts(tbase + Lay::kD, tbase + Lay::kQ + q * 32 + 8 * ks, dqt + (256 * ks >> 4), idD, f + (2 - q) + ks > 0);
              mma_bf16_ts(tbase + Lay::kD, tbase + Lay::kP + q * 32 + 8 * ks, dkt + (256 * ks >> 4), idD, 1);
            }
          if (f == 1) mma_commit(&bars[kDoneD]);
        }
        __syncwarp();
      }
      if (++s == Lay::kStages) s = 0, ++turn;
    }
  issued_all:
    if (chunks > 0) {
      if (elect_one()) mma_commit(&bars[kEnd]);
      __syncwarp();
      wait_own(&bars[kEnd], 0, a.err);
    }
  } else {
    const int quarter = warp & 3, up = warp >> 2;
    const int row = PM == 128 ? 32 * quarter + lane : 16 * quarter + (lane & 15);
    const int part = PM == 128 ? up : 2 * up + (lane >> 4);
    const int wpart = PM == 128 ? up : 2 * up;
    const uint32_t tq = tbase + ((uint32_t)(32 * quarter) << 16);
    const uint32_t tZ = tq + Lay::kZ + wpart * W, tA = tq + Lay::kA + wpart * W;
    const uint32_t tR = tq + Lay::kD + wpart * (W / 2), tU = tq + Lay::kP + wpart * (W / 2), tQ = tq + Lay::kQ + wpart * (W / 2),
                   tY = tq + Lay::kY + wpart * (W / 2);
    const uint32_t tX = tq + Lay::kP + wpart * (WN / 2), tD = tq + Lay::kD + wpart * WN;
    const int p = p0 + row, c0 = part * W, n0 = part * WN;
    const bool pin = p < a.P;
    const int N = (int)a.N;
    __nv_bfloat16 *dv = static_cast<__nv_bfloat16 *>(a.dv) + (b * a.L * a.H + h) * a.P + p;
    const int64_t step = a.H * a.P;
    float st[WN];
#pragma unroll
    for (int n = 0; n < WN; ++n) st[n] = (a.dh_final && pin && n0 + n < N) ? a.dh_final[(bh * a.N + n0 + n) * a.P + p] : 0.f;
    const auto ready = [&](int which) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[which]);
    };
    // dY of turn i as it is, an operand of dY^T A
    const auto store_dy = [&](int s, int turn) {
      if (!wait(kFull + s, turn & 1)) return false;
      const uint16_t *dy = reinterpret_cast<const uint16_t *>(smem + s * Lay::kStage + Lay::kDyOff) + c0 * PM + row;
      uint32_t r[W / 2];
#pragma unroll
      for (int c = 0; c < W / 2; ++c) r[c] = dy[2 * c * PM] | ((uint32_t)dy[(2 * c + 1) * PM] << 16);
      TmemIo<PM, W / 2>::st(tY, r);
      return true;
    };
    if (chunks > 0) {
      store_parts<PM, WN, 3>(tX, NP / 2, st);
      if (!store_dy(0, 0)) goto state_done;
      ready(kX + up);
    }
    for (int i = 0, s = 0, next = 0, turn = 0; i < chunks; ++i, s = next) {
      const int chunk = chunks - 1 - i;
      const uint32_t ph = i & 1;
      const uint8_t *stage = smem + s * Lay::kStage;
      const float *scal = reinterpret_cast<const float *>(stage + Lay::kRecOff + Lay::kRec - kScalars);
      const __nv_bfloat16 *dy = reinterpret_cast<const __nv_bfloat16 *>(stage + Lay::kDyOff) + c0 * PM + row;
      store_rows<PM, WN>(a.xcarry + ((bh * a.nC + chunk) * a.N + n0) * a.Pp + p, a.Pp, p < a.Pp ? N - n0 : 0, st);
      if (!wait(kDoneS, ph)) goto state_done;
      tc_fence_after();
      float x[W], w[W];
      load_cols<PM, W>(tZ, x);
      load_scalars<W>(w, scal + kChunk + c0);
#pragma unroll
      for (int c = 0; c < W; ++c) x[c] *= w[c];
      load_cols<PM, W>(tA, w);
#pragma unroll
      for (int c = 0; c < W; ++c) x[c] += w[c];
      store_parts<PM, W, 3>(tR, 32, x);
      ready(kR + up);
      // meanwhile scale dY diag(exp G); X's parts, whose place it may take, have been read
      load_scalars<W>(w, scal + c0);
#pragma unroll
      for (int c = 0; c < W; ++c) x[c] = a.scale * w[c] * __bfloat162float(dy[c * PM]);
      store_parts<PM, W, 3>(tQ, 32, x);
      if (!wait(kDoneU, ph)) goto state_done;
      tc_fence_after();
      load_cols<PM, W>(tZ, x);
      float g[W];
      load_scalars<W>(w, scal + 2 * kChunk + c0);
      load_scalars<W>(g, scal + c0);
#pragma unroll
      for (int c = 0; c < W; ++c) {
        w[c] *= x[c];
        g[c] *= -w[c];
      }
      store_parts<PM, W, 3>(tU, 32, g);
      ready(kU + up);
      {
        const int64_t t = (int64_t)chunk * kChunk + c0;
        const int n = (int)min((int64_t)W, len - t);
        __nv_bfloat16 *tv = dv + t * step;
        store_rows<PM, W>(a.du + (bh * a.L + t) * a.Pp + p, a.Pp, p < a.Pp ? n : 0, x);
        if (pin && n >= W) {
#pragma unroll
          for (int c = 0; c < W; ++c, tv += step) *tv = __float2bfloat16_rn(w[c]);
        } else if (pin) {
#pragma unroll
          for (int c = 0; c < W; ++c, tv += step)
            if (c < n) *tv = __float2bfloat16_rn(w[c]);
        }
      }
      const float last = scal[3 * kChunk], rest = scal[3 * kChunk + 1];
      if (!wait(kDoneD, ph)) goto state_done;
      tc_fence_after();
      {
        float d[WN];
        if constexpr (WN == 64) {
          load_cols<PM, 32>(tD, *reinterpret_cast<float(*)[32]>(d));
          load_cols<PM, 32>(tD + 32, *reinterpret_cast<float(*)[32]>(d + 32));
        } else {
          load_cols<PM, WN>(tD, d);
        }
#pragma unroll
        for (int n = 0; n < WN; ++n) st[n] = fmaf(last, st[n], fmaf(rest, st[n], d[n]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kFree + s]);
      if (++next == Lay::kStages) next = 0, ++turn;
      if (i + 1 < chunks) {
        store_parts<PM, WN, 3>(tX, NP / 2, st);
        if (!store_dy(next, turn)) goto state_done;
        ready(kX + up);
      }
    }
  state_done:
    tmem_wait_st();
    if (pin) {
      for (int64_t t = len + part; t < a.L; t += Lay::kParts) dv[t * step] = __float2bfloat16_rn(0.f);
      if (a.dh0) {
#pragma unroll
        for (int n = 0; n < WN; ++n)
          if (n0 + n < N) a.dh0[(bh * a.N + n0 + n) * a.P + p] = st[n];
      }
    }
  }
  tc_fence_before();
  const bool bad = __syncthreads_or(timed_out(a.err));
  if (warp == kIssuer) tmem_dealloc(tbase, Lay::kCols);
  if (bad && len > 0) {
    fill_nan(a.dv, true, (b * a.L * a.H + h) * a.P + p0, len, a.H * a.P, (int)min((int64_t)PM, a.P - p0), threadIdx.x, blockDim.x);
    fill_nan(a.dh0, false, bh * a.N * a.P + p0, a.N, a.P, (int)min((int64_t)PM, a.P - p0), threadIdx.x, blockDim.x);
  }
}

}  // namespace chunk_bwd
}  // namespace pdssm
