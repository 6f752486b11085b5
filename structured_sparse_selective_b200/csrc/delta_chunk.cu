// The gated delta rule by chunks of 64 steps, second part: the state from chunk to
// chunk and the outputs, one block per (sequence, head) (bf16 inputs; the records of
// csrc/delta_prep.cu; formulas in delta.cuh).
//
// For one chunk that starts from H, in the transposed form the tensor cores work on
// (rows are the value's columns p, M = 64 or 128 of them):
//   S = H^T K^T                       E = (V^T - S diag(exp G)) Te^T      u = beta e
//   H'^T = exp(G_64) H^T + (u exp(G_64 - G))^T K
//   Y^T = scale (H^T Q^T) diag(exp G) + U^T A^T
// Everything left of a product comes from tensor memory, where a thread has one row p
// (or a piece of it) and writes what it just computed; everything right of it is K, Q,
// Te or A in shared memory, K and Q read as [steps][n] for the first products and as
// [n][steps] for the update from the same bytes.
//
// Precision. K, Q, V are bf16 and exact. What is fp32 (H, R, u) is split into bf16 parts
// that are multiplied one by one and summed in fp32: three parts (24 bits) on the way to
// the state, so that it is an fp32 state; two parts (16 bits) where only y is
// reached, which is rounded to bf16 itself.
// SAVE (the forward of a backward pass) keeps three everywhere, since gradients of the
// gates are sums of <dy, y> in fp32; it writes these, e and the states instead of y. The
// products of small parts come first: an accumulator that is still small loses less when
// they are added to it.
//
// The chain K H -> Te -> K^T u is what a sequence waits for; it runs once a chunk, and the
// other products fill the pipe in its pauses. A product starts on the half of its depth
// that four of the eight state warps have written, while the others still write. Roles (12 warps): 8 keep the state (fp32, in
// registers: a row's n-range each) and do all elementwise work, a ninth issues the
// products, two bring K, Q (16-byte cp.async into the operand order), V and the record
// (bulk copies) ahead into two or three stages, and one writes y from shared memory.
// Every wait is bounded; when one has run out all roles leave their loops, and copies and products in
// flight are waited for before tensor memory is freed and the block ends.
// Measured: 256 sequences of 2,048 steps, 64 x 64: 150 us (two rounds of blocks, 4,600 cycles a chunk of 64
// steps), 128 of 4,096 steps, 128 x 128: 305 us (one round, 9,400 cycles): the chain of three products, each with
// its way through registers, is what a chunk takes. SAVE takes 230 and 465 us: the state's warps store the state
// and e and sum <dy, y> between one answer and the next. The kernels of 128 x 128 spill 104 to 164 bytes a thread.
#include <algorithm>

#include "delta.cuh"
#include "delta_chunk.cuh"
#include "delta_chunk_bwd.cuh"
#include "sm100.cuh"

namespace pdssm {

using namespace sm100;

namespace {

constexpr int kStateWarps = 8, kIssuer = 8, kLoader0 = 9, kLoaders = 2, kWriter = 11;
constexpr int kThreads = 32 * (kWriter + 1);

// kH, kR, kU: [half], from the four warps that have that half of a row's columns.
enum Bar { kFull, kFree = kFull + 3, kH = kFree + 3, kR = kH + 2, kU1 = kR + 2, kU2 = kU1 + 2, kRead, kDoneS, kDoneU, kDoneD, kDoneY, kOut, kOutFree, kDyFull, kDyFree, kEnd, kBars };

template <int NP, int PM, bool SAVE>
struct Layout {
  // tensor memory, 32-bit columns: X holds the state's parts (K H and Q H read them), then
  // u's parts; D the parts of R, then the update; Z has S, Ya first E, then U^T A^T. (E may
  // not take S's place: its product starts while half of the warps still read S.)
  static constexpr int kX = 0, kXn = 3 * NP / 2;
  static constexpr int kD = kXn, kDn = NP > 96 ? NP : 96;
  static constexpr int kYh = kD + kDn, kYa = kYh + 64, kZ = kYa + 64;
  static constexpr int kUd = kX;                                 // u exp(G_64 - G), three parts
  static constexpr int kUy = NP == 128 ? kX + 96 : kZ + 64;      // u, two or three parts
  static constexpr int kUyn = SAVE ? 96 : 64;
  static constexpr int kCols = 512;
  static_assert(kZ + 64 <= kCols && (NP == 128 || kUy + kUyn <= kCols) && (NP < 128 || 96 + kUyn <= kXn), "columns");
  // shared memory of a stage
  static constexpr int kRec = (3 + delta_a_parts(SAVE)) * kSquare + kScalars;
  static constexpr int kQ = (NP / 8) * kChunkGroup, kV = kChunk * PM * 2;  // V and Y: [step][p]
  static constexpr int kVOff = 2 * kQ, kRecOff = kVOff + kV, kStage = kRecOff + kRec;
  // three stages where they fit: loads have then two chunks' time; behind them y, or (SAVE) dY
  static constexpr int kY = kV, kStages = 3 * kStage + kY + 256 <= 227 * 1024 ? 3 : 2;
  static constexpr int kYOff = kStages * kStage, kBarOff = kYOff + kY, kBytes = kBarOff + 8 * kBars + 16;
  // a thread's share of a row: W of 64 steps, WN of NP state values
  static constexpr int kParts = 256 / PM, W = kChunk / kParts, WN = NP / kParts;
};

// One sequence of one head, columns p0 ...
template <int NP, int PM, bool SAVE>
__device__ __forceinline__ void run(const DeltaArgs &a, bool wide, bool wide_v, int p0) {
  using Lay = Layout<NP, PM, SAVE>;
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
      const bool half = i >= kH && i < kU2, state = (i >= kFree && i < kH) || i == kU2 || i == kRead || i == kOut || i == kDyFree;
      mbar_init(&bars[i], half ? kStateWarps / 2 : state ? kStateWarps : i < kFree ? 32 * kLoaders + 1 : i == kDyFull ? 32 * kLoaders : 1);
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

  if (warp == kWriter) {
    if (!SAVE) {
      // y of a chunk: from [step][p] in shared memory, 16 bytes a lane
      __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + (b * a.L * a.H + h) * a.P + p0;
      const int64_t step = a.H * a.P;
      const uint8_t *tile = smem + Lay::kYOff;
      const int P = (int)min((int64_t)PM, a.P - p0);
      for (int i = 0; i < chunks; ++i) {
        if (!wait(kOut, i & 1)) break;
        const int live = (int)min((int64_t)kChunk, len - (int64_t)i * kChunk);
        __nv_bfloat16 *dst = y + (int64_t)i * kChunk * step;
        constexpr int G = PM / 8, kRows = 32 / G;
        const int g = lane % G;
#pragma unroll 4
        for (int c = lane / G; c < kChunk; c += kRows) {
          if (c >= live) continue;
          if (wide_v) {
            if (8 * g < P) *reinterpret_cast<uint4 *>(dst + c * step + 8 * g) = *reinterpret_cast<const uint4 *>(tile + (c * PM + 8 * g) * 2);
          } else {
            for (int k = 8 * g; k < min(P, 8 * g + 8); ++k) dst[c * step + k] = reinterpret_cast<const __nv_bfloat16 *>(tile)[c * PM + k];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kOutFree]);
      }
      for (int64_t t = len; t < a.L; ++t)
        for (int k = lane; k < P; k += 32) y[t * step + k] = __float2bfloat16_rn(0.f);
    }
  } else if (warp >= kLoader0) {
    const int tid = threadIdx.x - 32 * kLoader0;
    const bool copies = wide && wide_v && a.N == NP && a.P - p0 >= PM;  // nothing is written by the threads themselves
    using B = const __nv_bfloat16;
    const auto go_on = [&](int which, uint32_t parity) {
      return all_of<32 * kLoaders>(wait_bar(&bars[which], parity, a.err, a.wait_ns));
    };
    int issued = 0, dys = 0;
    // a short limit runs out here: nothing has been asked for yet
    if (a.wait_ns < kShortNs && chunks > 0) all_of<32 * kLoaders>(wait_slow<false>(&bars[kFull], 0, a.err, a.wait_ns));
    // SAVE: dY of chunk i, which is wanted at the chunk's end, comes behind the next chunk's stage
    const auto load_dy = [&](int i) {
      if (i >= 1 && !go_on(kDyFree, (i - 1) & 1)) return false;
      const int live = (int)min((int64_t)kChunk, len - (int64_t)i * kChunk);
      load_tile<PM / 8, 16, 2 * PM, 32 * kLoaders>(smem + Lay::kYOff, static_cast<B *>(a.dy), b * a.L + (int64_t)i * kChunk, a.H, h, a.P,
                                                   p0, live, wide_v, tid);
      if (copies && live == kChunk) {
        cp_async_arrive(&bars[kDyFull]);
      } else {
        cp_async_commit();
        cp_async_wait<0>();
        mbar_arrive(&bars[kDyFull]);
      }
      ++dys;
      return true;
    };
    for (int i = 0, s = 0, turn = 0; i < chunks; ++i) {
      if (turn && !go_on(kFree + s, (turn - 1) & 1)) break;
      uint8_t *st = smem + s * Lay::kStage;
      uint64_t *full = &bars[kFull + s];
      const int live = (int)min((int64_t)kChunk, len - (int64_t)i * kChunk);
      const int64_t row0 = b * a.L + (int64_t)i * kChunk;
      const bool whole = copies && live == kChunk;
      if (tid < 32) {
        const uint8_t *rec = a.records + (bh * a.nC + i) * a.rec_bytes;
        if (lane == 0) {
          mbar_expect_tx(full, Lay::kRec);
          if (SAVE) {  // the record has Tb between Te and A
            bulk_load(st + Lay::kRecOff, rec, 3 * kSquare, full);
            bulk_load(st + Lay::kRecOff + 3 * kSquare, rec + 6 * kSquare, 3 * kSquare + kScalars, full);
          } else {
            bulk_load(st + Lay::kRecOff, rec, Lay::kRec, full);
          }
        }
      }
      load_tile<NP / 8, kChunkGroup, 16, 32 * kLoaders>(st, static_cast<B *>(a.k), row0, a.Hk, hk, a.N, 0, live, wide, tid);
      load_tile<NP / 8, kChunkGroup, 16, 32 * kLoaders>(st + Lay::kQ, static_cast<B *>(a.q), row0, a.Hk, hk, a.N, 0, live, wide, tid);
      load_tile<PM / 8, 16, 2 * PM, 32 * kLoaders>(st + Lay::kVOff, static_cast<B *>(a.v), row0, a.H, h, a.P, p0, live, wide_v, tid);
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
      if (SAVE && i >= 1 && !load_dy(i - 1)) break;
    }
    if (SAVE && chunks > 0 && issued == chunks) load_dy(chunks - 1);
    if (SAVE && dys > 0) wait_own(&bars[kDyFull], (dys - 1) & 1, a.err);
    for (int i = max(issued - Lay::kStages, 0); i < issued; ++i) wait_own(&bars[kFull + i % Lay::kStages], (i / Lay::kStages) & 1, a.err);
  } else if (warp == kIssuer) {
    // The whole warp goes through the loop and one lane issues: descriptors and addresses
    // are then uniform (computed by one lane alone they cost about 70 cycles a product,
    // twice the product itself).
    constexpr uint32_t idS = idesc_bf16_f32(PM, kChunk, false, false), idD = idesc_bf16_f32(PM, NP, false, true);
    const uint32_t base = smem_u32(smem);
    for (int i = 0, s = 0, turn = 0; i < chunks; ++i) {
      const uint32_t ph = i & 1, sk = base + s * Lay::kStage, sq = sk + Lay::kQ, te = sk + Lay::kRecOff, sa = te + 3 * kSquare;
      const uint64_t dk = smem_desc(sk, kChunkGroup, 128), dq = smem_desc(sq, kChunkGroup, 128), dkt = smem_desc(sk, 128, kChunkGroup),
                     dte = smem_desc(te, 1024, 128), da = smem_desc(sa, 1024, 128);
      if (!wait(kFull + s, turn & 1)) goto issued_all;
      fence_proxy_async_smem();  // the loaders' writes, seen through the barrier, before the tensor core's reads
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        if (!wait(kH + f, ph)) goto issued_all;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int q = 2; q >= 0; --q)
#pragma unroll
            for (int ks = f * NP / 32; ks < (f + 1) * NP / 32; ++ks)
              mma_bf16_ts(tbase + Lay::kZ, tbase + Lay::kX + q * (NP / 2) + 8 * ks, dk + (2 * kChunkGroup * ks >> 4), idS, f + (2 - q) + ks > 0);
          if (f == 1) mma_commit(&bars[kDoneS]);
        }
        __syncwarp();
      }
      // Q H into Yh, once the chunk before has been read out of it
      if (i >= 1 && !wait(kRead, (i - 1) & 1)) goto issued_all;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int q = SAVE ? 2 : 1; q >= 0; --q)
#pragma unroll
          for (int ks = 0; ks < NP / 16; ++ks)
            mma_bf16_ts(tbase + Lay::kYh, tbase + Lay::kX + q * (NP / 2) + 8 * ks, dq + (2 * kChunkGroup * ks >> 4), idS,
                        (SAVE ? 2 : 1) - q + ks > 0);
      }
      __syncwarp();
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        if (!wait(kR + f, ph)) goto issued_all;
        tc_fence_after();
        if (elect_one()) {
          // R Te^T: parts (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
#pragma unroll
          for (int o = 2; o >= 0; --o)
#pragma unroll
            for (int q = 0; q <= o; ++q)
#pragma unroll
              for (int ks = 2 * f; ks < 2 * f + 2; ++ks)
                mma_bf16_ts(tbase + Lay::kYa, tbase + Lay::kD + (o - q) * 32 + 8 * ks, dte + ((q * kSquare + 2048 * ks) >> 4), idS,
                            f + (2 - o) + q + ks > 0);
          if (f == 1) mma_commit(&bars[kDoneU]);
        }
        __syncwarp();
      }
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        if (!wait(kU1 + f, ph)) goto issued_all;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int q = 2; q >= 0; --q)
#pragma unroll
            for (int ks = 2 * f; ks < 2 * f + 2; ++ks)
              mma_bf16_ts(tbase + Lay::kD, tbase + Lay::kUd + q * 32 + 8 * ks, dkt + (256 * ks >> 4), idD, f + (2 - q) + ks > 0);
          if (f == 1) mma_commit(&bars[kDoneD]);
        }
        __syncwarp();
      }
      if (!wait(kU2, ph)) goto issued_all;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int o = SAVE ? 2 : 1; o >= 0; --o)
#pragma unroll
          for (int q = 0; q <= o; ++q) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_bf16_ts(tbase + Lay::kYa, tbase + Lay::kUy + (o - q) * 32 + 8 * ks, da + ((q * kSquare + 2048 * ks) >> 4), idS,
                          (SAVE ? 2 : 1) - o + q + ks > 0);
          }
        mma_commit(&bars[kDoneY]);
      }
      __syncwarp();
      if (++s == Lay::kStages) s = 0, ++turn;
    }
  issued_all:
    if (chunks > 0) {
      if (elect_one()) mma_commit(&bars[kEnd]);
      __syncwarp();
      wait_own(&bars[kEnd], 0, a.err);
    }
  } else {
    // the state's warps
    const int quarter = warp & 3, up = warp >> 2;
    const int row = PM == 128 ? 32 * quarter + lane : 16 * quarter + (lane & 15);
    const int part = PM == 128 ? up : 2 * up + (lane >> 4);
    const int wpart = PM == 128 ? up : 2 * up;  // where the warp's accesses of a row begin, in parts
    const uint32_t tq = tbase + ((uint32_t)(32 * quarter) << 16);
    const uint32_t tZ = tq + Lay::kZ + wpart * W, tYh = tq + Lay::kYh + wpart * W, tYa = tq + Lay::kYa + wpart * W;
    const uint32_t tR = tq + Lay::kD + wpart * (W / 2), tUd = tq + Lay::kUd + wpart * (W / 2), tUy = tq + Lay::kUy + wpart * (W / 2);
    const uint32_t tX = tq + Lay::kX + wpart * (WN / 2), tD = tq + Lay::kD + wpart * WN;
    const int p = p0 + row, c0 = part * W, n0 = part * WN;
    const bool pin = p < a.P;
    const int N = (int)a.N;
    float st[WN];
#pragma unroll
    for (int n = 0; n < WN; ++n) st[n] = (a.h0 && pin && n0 + n < N) ? a.h0[(bh * a.N + n0 + n) * a.P + p] : 0.f;
    const auto ready = [&](int which) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[which]);
    };
    // SAVE: the state before chunk i (and behind the last), and 64 x p values of the chunk's steps
    const auto save_state = [&](int i) {
      store_rows<PM, WN>(a.carry + ((bh * (a.nC + 1) + i) * a.N + n0) * a.Pp + p, a.Pp, p < a.Pp ? N - n0 : 0, st);
    };
    const auto save_rows = [&](float *rows, int i, const float (&x)[W]) {
      const int64_t t = (int64_t)i * kChunk + c0;
      store_rows<PM, W>(rows + (bh * a.L + t) * a.Pp + p, a.Pp, p < a.Pp ? (int)min((int64_t)W, len - t) : 0, x);
    };
    // the thread's values of chunk i, two steps a register: read a product ahead of their use
    uint32_t vv[W / 2];
    const auto fetch_v = [&](int s, int turn) {
      if (!wait(kFull + s, turn & 1)) return false;
      const uint16_t *v = reinterpret_cast<const uint16_t *>(smem + s * Lay::kStage + Lay::kVOff) + c0 * PM + row;
#pragma unroll
      for (int c = 0; c < W / 2; ++c) vv[c] = v[2 * c * PM] | ((uint32_t)v[(2 * c + 1) * PM] << 16);
      return true;
    };
    // y of chunk i, rounded, two steps a register, and its way to the writer
    uint32_t yy[SAVE ? 1 : W / 2];
    const auto put_y = [&](int i) {
      if (i >= 1 && !wait(kOutFree, (i - 1) & 1)) return false;
      uint16_t *out = reinterpret_cast<uint16_t *>(smem + Lay::kYOff) + c0 * PM + row;
#pragma unroll
      for (int c = 0; c < (SAVE ? 1 : W / 2); ++c) {
        out[2 * c * PM] = (uint16_t)yy[c];
        out[(2 * c + 1) * PM] = (uint16_t)(yy[c] >> 16);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kOut]);
      return true;
    };
    if (chunks > 0) {
      if (!fetch_v(0, 0)) goto state_done;
      store_parts<PM, WN, 3>(tX, NP / 2, st);
      ready(kH + up);
    }
    for (int i = 0, s = 0, next = 0, turn = 0; i < chunks; ++i, s = next) {
      const uint32_t ph = i & 1;
      const uint8_t *stage = smem + s * Lay::kStage;
      const float *scal = reinterpret_cast<const float *>(stage + Lay::kRecOff + Lay::kRec - kScalars);
      if (SAVE) save_state(i);
      float x[W], w[W];
      load_scalars<W>(w, scal + c0);
      if (!wait(kDoneS, ph)) goto state_done;
      tc_fence_after();
      load_cols<PM, W>(tZ, x);
#pragma unroll
      for (int c = 0; c < W; ++c) x[c] = fmaf(-w[c], x[c], c & 1 ? high_half(vv[c / 2]) : low_half(vv[c / 2]));
      store_parts<PM, W, 3>(tR, 32, x);
      ready(kR + up);
      if (!SAVE && i >= 1 && !put_y(i - 1)) goto state_done;
      load_scalars<W>(w, scal + 2 * kChunk + c0);
      if (!wait(kDoneU, ph)) goto state_done;
      tc_fence_after();
      load_cols<PM, W>(tYa, x);
#pragma unroll
      for (int c = 0; c < W; ++c) x[c] *= w[c];
      load_scalars<W>(w, scal + kChunk + c0);
#pragma unroll
      for (int c = 0; c < W; ++c) w[c] *= x[c];
      store_parts<PM, W, 3>(tUd, 32, w);
      ready(kU1 + up);
      store_parts<PM, W, SAVE ? 3 : 2>(tUy, 32, x);
      if (SAVE) {  // e is still in its accumulator: read again, behind what the chain waits for
        float e[W];
        load_cols<PM, W>(tYa, e);
        ready(kU2);
        save_rows(a.e, i, e);
      } else {
        ready(kU2);
      }
      if (++next == Lay::kStages) next = 0, ++turn;
      if (i + 1 < chunks && !fetch_v(next, turn)) goto state_done;
      if (!wait(kDoneD, ph)) goto state_done;
      tc_fence_after();
      const float last = scal[3 * kChunk], rest = scal[3 * kChunk + 1];
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
      // where u's parts lie among those of the state, the product with A has to be done too
      if (Lay::kUy < Lay::kD) {
        if (!wait(kDoneY, ph)) goto state_done;
        tc_fence_after();
      }
      if (i + 1 < chunks) {
        store_parts<PM, WN, 3>(tX, NP / 2, st);
        ready(kH + up);
      }
      if (Lay::kUy >= Lay::kD) {
        if (!wait(kDoneY, ph)) goto state_done;
        tc_fence_after();
      }
      // y's scalars are read before the stage goes back to the loaders
      float g[W];
      load_scalars<W>(g, scal + c0);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kFree + s]);
      load_cols<PM, W>(tYa, w);
      load_cols<PM, W>(tYh, x);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kRead]);
#pragma unroll
      for (int c = 0; c < W; ++c) x[c] = fmaf(a.scale * g[c], x[c], w[c]);
      if (SAVE) {
        // <dy, y> of the warp's columns of p: products summed over its rows, a lane ends with one step's
        if (!wait(kDyFull, ph)) goto state_done;
        const __nv_bfloat16 *dy = reinterpret_cast<const __nv_bfloat16 *>(smem + Lay::kYOff) + c0 * PM + row;
#pragma unroll
        for (int c = 0; c < W; ++c) x[c] *= __bfloat162float(dy[c * PM]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kDyFree]);
#pragma unroll
        for (int o = W / 2; o >= 1; o >>= 1) {
          const bool upper = lane & o;
#pragma unroll
          for (int c = 0; c < o; ++c) {
            const float mine = upper ? x[c + o] : x[c], other = upper ? x[c] : x[c + o];
            x[c] = mine + __shfl_xor_sync(0xffffffffu, other, o);
          }
        }
        const int64_t t = (int64_t)i * kChunk + c0 + (lane & (W - 1));
        if (t < len) a.dyy[(bh * a.L + t) * 4 + quarter] = x[0];
      } else {
        // y goes to the writer in the next chunk's first pause, or at once behind the last
#pragma unroll
        for (int c = 0; c < W / 2; ++c) yy[c] = pack_bf16(x[2 * c], x[2 * c + 1]);
        if (i + 1 == chunks && !put_y(i)) goto state_done;
      }
    }
  state_done:
    tmem_wait_st();
    if (SAVE) save_state(chunks);
    if (!SAVE && pin && a.h_final) {
#pragma unroll
      for (int n = 0; n < WN; ++n)
        if (n0 + n < N) a.h_final[(bh * a.N + n0 + n) * a.P + p] = st[n];
    }
  }
  tc_fence_before();
  const bool bad = __syncthreads_or(timed_out(a.err));
  if (warp == kIssuer) tmem_dealloc(tbase, Lay::kCols);
  if (!SAVE && bad && len > 0) {
    fill_nan(a.y, true, (b * a.L * a.H + h) * a.P + p0, len, a.H * a.P, (int)min((int64_t)PM, a.P - p0), threadIdx.x, kThreads);
    fill_nan(a.h_final, false, bh * a.N * a.P + p0, a.N, a.P, (int)min((int64_t)PM, a.P - p0), threadIdx.x, kThreads);
  }
}

enum What { kForward, kSave, kBack, kBoth };

// kBoth: the states and the adjoints of a backward pass do not need one another, so their blocks
// take turns in one launch.
template <int NP, int PM, What WHAT>
__global__ void __launch_bounds__(kThreads, 1) delta_chunk_kernel(DeltaArgs a, bool wide, bool wide_v) {
  const int p0 = (WHAT == kBoth ? blockIdx.x >> 1 : blockIdx.x) * PM;
  if (WHAT == kBack || (WHAT == kBoth && (blockIdx.x & 1))) chunk_bwd::run<NP, PM>(a, wide, wide_v, p0);
  else run<NP, PM, WHAT != kForward>(a, wide, wide_v, p0);
}

bool all16(const void *x, const void *y) {
  return ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & 15) == 0;
}

template <int NP, int PM, What WHAT>
cudaError_t launch_k(const DeltaArgs &a, const char *name, cudaStream_t st) {
  auto kern = delta_chunk_kernel<NP, PM, WHAT>;
  constexpr int kSave_ = Layout<NP, PM, true>::kBytes, kBack_ = chunk_bwd::Layout<NP, PM>::kBytes;
  constexpr int kSmem = WHAT == kForward ? Layout<NP, PM, false>::kBytes
                        : WHAT == kSave  ? kSave_
                        : WHAT == kBack  ? kBack_
                        : kSave_ > kBack_ ? kSave_ : kBack_;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess || (e = trace_before(st, name)) != cudaSuccess) return e;
  const bool wide = a.N % 8 == 0 && all16(a.q, a.k), wide_v = a.P % 8 == 0 && all16(a.v, WHAT == kForward ? a.y : a.dy);
  const dim3 grid((unsigned)((a.P + PM - 1) / PM) * (WHAT == kBoth ? 2 : 1), (unsigned)a.H, (unsigned)a.Bt);
  kern<<<grid, kThreads, kSmem, st>>>(a, wide, wide_v);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : trace_after(st);
}

template <int NP, int PM>
cudaError_t launch_n(const DeltaArgs &a, bool bwd, cudaStream_t st) {
  if (!bwd) return launch_k<NP, PM, kForward>(a, "delta_chunk", st);
  // One launch where all its blocks have an SM of their own (64 sequences of 2,048 steps, 128 x 128: 304 us
  // together, 412 one after the other); beyond that the two kinds slow one another (256 sequences, 64 x 64:
  // 490 and 424 us; 128 of 4,096 steps, 128 x 128: 1,078 and 834).
  if (2 * a.Bt * a.H * ((a.P + PM - 1) / PM) <= 148) return launch_k<NP, PM, kBoth>(a, "delta_chunk_both", st);
  cudaError_t e = launch_k<NP, PM, kSave>(a, "delta_chunk_save", st);
  return e != cudaSuccess ? e : launch_k<NP, PM, kBack>(a, "delta_chunk_bwd", st);
}

cudaError_t launch(const DeltaArgs &a, bool bwd, cudaStream_t st) {
  if (a.N <= 64) return a.P <= 64 ? launch_n<64, 64>(a, bwd, st) : launch_n<64, 128>(a, bwd, st);
  return a.P <= 64 ? launch_n<128, 64>(a, bwd, st) : launch_n<128, 128>(a, bwd, st);
}

}  // namespace

cudaError_t launch_delta_chunk(const DeltaArgs &a, cudaStream_t st) { return launch(a, false, st); }
cudaError_t launch_delta_chunk_both(const DeltaArgs &a, cudaStream_t st) { return launch(a, true, st); }

}  // namespace pdssm
