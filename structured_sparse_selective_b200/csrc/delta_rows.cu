// The gated delta rule by chunks of 32 steps in fp32 (fp32 inputs), forwards and backwards.
//
// With G the sums of the gates within a chunk, D_ij = exp(G_i - G_j), N_ij = D_ij <k_i, k_j> (j < i),
// A_ij = scale D_ij <q_i, k_j> (j <= i), X = (1 + N diag beta)^-1 N and the state H before the chunk:
//   E = Te (V - diag(exp G) K H),  Te = 1 - X diag beta,   U = diag(beta) E
//   Y = scale diag(exp G) Q H + A U
//   H' = exp(G_32) H + K^T diag(exp(G_32 - G)) U
// and for the adjoint X of the state behind the chunk:
//   dU = Tb^T (diag(exp(G_32 - G)) K X + A^T dY),  Tb = 1 - diag(beta) X,   dV = diag(beta) dU
//   X' = exp(G_32) X + scale Q^T diag(exp G) dY - K^T diag(exp G) dV
// A first kernel makes what does not depend on the state: Te (Tb^T), A (A^T) and the scalars of every
// chunk of every value head, and K, K^T, Q (Q^T) of every key head in the order the lanes read them.
//
// The columns p are independent of one another, so in the second kernel a warp has CW of them and
// goes through the chunks on its own, without a barrier between warps: the left operand's rows
// (steps; rows of the state) lie on the lanes, the right one's values are broadcast from the warp's
// own shared memory, two terms of a sum an instruction (fma.rn.f32x2). One warp more asks for the
// records, a bulk copy each, up to three chunks ahead; in blocks of eight, whose registers leave no room
// for a ninth, the first warp does, which waits for the others for it (32 sequences of 18,000 steps,
// 32 x 32: 650 us so, 545 with the warp more; two blocks instead of eight warps make a second round of
// blocks: 2 x 2,048 steps x 32 heads of 128 x 128 took 1,035 us in blocks of six, 690 in blocks of eight).
// What bounds it: with few sequences the five products' latencies, one after the other (about 1,850
// cycles a chunk of 32 steps, against 5,000 for 32 steps by csrc/delta_steps.cu); with many the FMA pipe
// and the shared-memory reads (a broadcast and a quarter of a row read for every 2 x CW FMAs).
#include <algorithm>

#include "delta.cuh"
#include "delta_chunk.cuh"
#include "sm100.cuh"

namespace pdssm {

using namespace sm100;

namespace {

constexpr int kC = 32;        // steps a chunk
constexpr int kTri = kC * kC;  // values of a triangle
constexpr int kScal = 4 * kC;  // exp G, exp(G_32 - G), beta, exp(G_32) in two parts

// Values of a record. A key head's: K [n / 4][step][4], K^T [step / 4][n][4], then Q as K, or
// (backward) Q^T as K^T. A value head's: Te [j / 4][step][4], the scalars, then A as Te, or
// (backward) Tb^T [i / 4][j][4] and A^T.
__host__ __device__ constexpr int key_values(int NP) { return 3 * kC * NP; }
__host__ __device__ constexpr int head_values(bool bwd) { return (bwd ? 3 : 2) * kTri + kScal; }

// ------------------------------------------------------------------ records

constexpr int kPrepWarps = 4, kGroup = 4 * kC + 4, kLd = kC + 4;  // groups of four columns, rows of a triangle; padded

template <int NP>
constexpr int prep_values() { return 2 * (NP / 4) * kGroup > 2 * kC * kLd ? 2 * (NP / 4) * kGroup : 2 * kC * kLd; }

// A warp has one chunk of one key head and the value heads that share it.
template <int NP, bool BWD>
__global__ void __launch_bounds__(32 * kPrepWarps, BWD ? 2 : 4) delta_rows_prep_kernel(DeltaArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *ks = reinterpret_cast<float *>(smem) + warp * prep_values<NP>(), *qs = ks + (NP / 4) * kGroup;
  float *nt = ks, *tt = ks + kC * kLd;  // in the place of K and Q once their products are known
  const int64_t chunk = (int64_t)blockIdx.x * kPrepWarps + warp, hk = blockIdx.y, b = blockIdx.z, t0 = chunk * kC;
  const int64_t len = live_steps(a.lengths, b, a.L);
  if (t0 >= len) return;
  const int live = (int)min((int64_t)kC, len - t0), N = (int)a.N;
  const float *k0 = static_cast<const float *>(a.k) + ((b * a.L + t0) * a.Hk + hk) * N;
  const float *q0 = static_cast<const float *>(a.q) + ((b * a.L + t0) * a.Hk + hk) * N;
  const int64_t step = a.Hk * N;
#pragma unroll
  for (int j = 0; j < NP / 32; ++j) {
    const int n = 32 * j + lane, nn = min(n, N - 1);
    const bool in = n < N;
#pragma unroll 16
    for (int t = 0; t < kC; ++t) {
      const int64_t at = (int64_t)min(t, live - 1) * step + nn;
      const float kv = k0[at], qv = q0[at];
      const bool on = in && t < live;
      ks[(n >> 2) * kGroup + 4 * t + (n & 3)] = on ? kv : 0.f;
      qs[(n >> 2) * kGroup + 4 * t + (n & 3)] = on ? qv : 0.f;
    }
  }
  __syncwarp();
  float *key = a.keys + ((b * a.Hk + hk) * a.nC + chunk) * key_values(NP);
#pragma unroll 4
  for (int g = 0; g < NP / 4; ++g) {
    reinterpret_cast<float4 *>(key)[g * 32 + lane] = *reinterpret_cast<const float4 *>(ks + g * kGroup + 4 * lane);
    if (!BWD) reinterpret_cast<float4 *>(key + 2 * kC * NP)[g * 32 + lane] = *reinterpret_cast<const float4 *>(qs + g * kGroup + 4 * lane);
  }
#pragma unroll 2
  for (int i = 0; i < NP / 4; ++i) {  // eight groups of steps, NP / 32 of rows
    const int g = i / (NP / 32), n = 32 * (i % (NP / 32)) + lane;
    const auto column = [&](const float *s) {
      const float *p = s + (n >> 2) * kGroup + 16 * g + (n & 3);
      return make_float4(p[0], p[4], p[8], p[12]);
    };
    reinterpret_cast<float4 *>(key + kC * NP)[g * NP + n] = column(ks);
    if (BWD) reinterpret_cast<float4 *>(key + 2 * kC * NP)[g * NP + n] = column(qs);
  }
  // rows of K K^T and Q K^T, a row a lane
  float kk[kC] = {}, qk[kC] = {};
#pragma unroll 1
  for (int g = 0; g < NP / 4; ++g) {
    const float4 x = *reinterpret_cast<const float4 *>(ks + g * kGroup + 4 * lane), y = *reinterpret_cast<const float4 *>(qs + g * kGroup + 4 * lane);
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const float4 z = *reinterpret_cast<const float4 *>(ks + g * kGroup + 4 * j);
      kk[j] = fmaf(x.x, z.x, fmaf(x.y, z.y, fmaf(x.z, z.z, fmaf(x.w, z.w, kk[j]))));
      qk[j] = fmaf(y.x, z.x, fmaf(y.y, z.y, fmaf(y.z, z.z, fmaf(y.w, z.w, qk[j]))));
    }
  }
  const int r = (int)(a.H / a.Hk);
  const bool gb = a.gate_t == PDSSM_BF16;
  for (int hh = 0; hh < r; ++hh) {
    const int64_t h = hk * r + hh, at = (b * a.L + t0 + min(lane, live - 1)) * a.H + h;
    float *rec = a.heads + ((b * a.H + h) * a.nC + chunk) * head_values(BWD);
    // sums of the gates in double, as two floats
    const double g0 = lane < live ? (double)clamp_gate(load_any(a.g, at, gb)) * 1.4426950408889634 : 0.0;
    const float beta = lane < live ? load_any(a.beta, at, gb) : 0.f;
    double sum = g0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    const double last = __shfl_sync(0xffffffffu, sum, 31);
    const float hi = (float)sum, lo = (float)(sum - (double)hi);
    rec[kTri + lane] = decay2(hi);
    rec[kTri + kC + lane] = decay2((float)(last - sum));
    rec[kTri + 2 * kC + lane] = beta;
    // the state's decay over the chunk, as a float and what that lacks: hundreds of them are multiplied
    const double all = exp2(last);
    rec[kTri + 3 * kC + lane] = lane & 1 ? (float)(all - (double)(float)all) : (float)all;
    __syncwarp();  // nt and tt: the head before has been read, or K and Q
    float row[kC];
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const float d = decay2((hi - __shfl_sync(0xffffffffu, hi, j)) + (lo - __shfl_sync(0xffffffffu, lo, j)));
      nt[j * kLd + lane] = j < lane ? d * kk[j] : 0.f;
      row[j] = j <= lane ? a.scale * d * qk[j] : 0.f;
      if (BWD) tt[j * kLd + lane] = row[j];
    }
    if (!BWD) {
#pragma unroll
      for (int g = 0; g < kC / 4; ++g)
        reinterpret_cast<float4 *>(rec + kTri + kScal)[g * 32 + lane] = make_float4(row[4 * g], row[4 * g + 1], row[4 * g + 2], row[4 * g + 3]);
    }
    __syncwarp();
    if (BWD) {
#pragma unroll
      for (int g = 0; g < kC / 4; ++g)
        reinterpret_cast<float4 *>(rec + 2 * kTri + kScal)[g * 32 + lane] = *reinterpret_cast<const float4 *>(tt + lane * kLd + 4 * g);
    }
    // column `lane` of X by forward substitution: each known value is taken out of the rows below it
    float x[kC];
#pragma unroll
    for (int g = 0; g < kC / 4; ++g) {
      const float4 v = *reinterpret_cast<const float4 *>(nt + lane * kLd + 4 * g);
      x[4 * g] = v.x; x[4 * g + 1] = v.y; x[4 * g + 2] = v.z; x[4 * g + 3] = v.w;
    }
#pragma unroll
    for (int m = 1; m < kC - 1; ++m) {
      const float xm = -__shfl_sync(0xffffffffu, beta, m) * x[m];
#pragma unroll
      for (int g = (m + 1) / 4; g < kC / 4; ++g) {
        const float4 v = *reinterpret_cast<const float4 *>(nt + m * kLd + 4 * g);
        const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int s = 0; s < 4; ++s)
          if (4 * g + s > m) x[4 * g + s] = fmaf(w[s], xm, x[4 * g + s]);
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kC; ++i) tt[i * kLd + lane] = i > lane ? -beta * x[i] : i == lane ? 1.f : 0.f;
    __syncwarp();
#pragma unroll
    for (int g = 0; g < kC / 4; ++g)
      reinterpret_cast<float4 *>(rec)[g * 32 + lane] = *reinterpret_cast<const float4 *>(tt + lane * kLd + 4 * g);
    if (BWD) {
#pragma unroll
      for (int i = 0; i < kC; ++i) row[i] = -__shfl_sync(0xffffffffu, beta, i) * x[i];
#pragma unroll
      for (int g = 0; g < kC / 4; ++g) {
        float w[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) w[s] = 4 * g + s > lane ? row[4 * g + s] : 4 * g + s == lane ? 1.f : 0.f;
        reinterpret_cast<float4 *>(rec + kTri + kScal)[g * 32 + lane] = make_float4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// ------------------------------------------------------------------ chunk after chunk

enum What { kForward, kSave, kBack };

// Right operands of a warp's products in shared memory, value (row, column c): (row / 2) * LD + 2 * c + row % 2,
// so a read has two rows' values of two columns; LD is padded for the writes.
template <int CW>
struct Warp {
  static constexpr int LD = 2 * CW + 4;
  static constexpr int values(int NP, What what) { return (NP / 2 + (what == kBack ? 4 : what == kSave ? 2 : 3) * kC / 2) * LD; }
};

// acc[c] += two partial sums over 4 GROUPS terms of rows[g] (four terms of the lane's row) and bc.
// A batch of groups is read while the one before is multiplied (left to the compiler, each group
// waited for its reads: 32 sequences of 18,000 steps, 32 x 32, took 1,137 instead of 697 us), no more
// than eight groups are unrolled (more, and the reads of several products at once spilled registers:
// 2 x 2,048 steps x 32 heads of 128 x 128 backwards 3,120 instead of 1,555 us).
template <int CW, int GROUPS>
__device__ __forceinline__ void mul_block(const float4 *rows, int stride, const float *bc, pair2 (&acc)[CW]) {
  constexpr int LD = Warp<CW>::LD, B = 8 / CW, BATCHES = GROUPS / B;
  float4 k[2][B], x[2][B][2][CW / 2];
  const auto read = [&](int b, int to) {
#pragma unroll
    for (int g = 0; g < B; ++g) {
      k[to][g] = rows[(b * B + g) * stride];
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int i = 0; i < CW / 2; ++i) x[to][g][half][i] = reinterpret_cast<const float4 *>(bc + (2 * (b * B + g) + half) * LD)[i];
    }
  };
  read(0, 0);
#pragma unroll
  for (int b = 0; b < BATCHES; ++b) {
    if (b + 1 < BATCHES) read(b + 1, (b + 1) & 1);
#pragma unroll
    for (int g = 0; g < B; ++g)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float4 w = k[b & 1][g];
        const pair2 kk = half ? pack2(w.z, w.w) : pack2(w.x, w.y);
#pragma unroll
        for (int i = 0; i < CW / 2; ++i) {
          const float4 v = x[b & 1][g][half][i];
          acc[2 * i] = fma2(kk, pack2(v.x, v.y), acc[2 * i]);
          acc[2 * i + 1] = fma2(kk, pack2(v.z, v.w), acc[2 * i + 1]);
        }
      }
  }
}
template <int CW, int GROUPS>
__device__ __forceinline__ void mul(const float4 *rows, int stride, const float *bc, pair2 (&acc)[CW]) {
#pragma unroll 1
  for (int g = 0; g < GROUPS; g += 8) mul_block<CW, 8>(rows + g * stride, stride, bc + 2 * g * Warp<CW>::LD, acc);
  __syncwarp();  // keeps the next product's reads, and their registers, behind this one
}

template <int CW>
__device__ __forceinline__ void put(float *bc, int row, const float (&v)[CW]) {
  float *p = bc + (row >> 1) * Warp<CW>::LD + (row & 1);
#pragma unroll
  for (int c = 0; c < CW; ++c) p[2 * c] = v[c];
}

__device__ __forceinline__ float both(pair2 v) {
  float x, y;
  unpack2(v, x, y);
  return x + y;
}

// The first `n` of CW columns at p, zeros behind them; aligned: by 16 bytes (8 for two columns).
template <int CW>
__device__ __forceinline__ void load_cols_f32(float (&v)[CW], const float *p, int n, bool aligned) {
  if (!aligned) {
#pragma unroll
    for (int c = 0; c < CW; ++c) v[c] = c < n ? p[c] : 0.f;
  } else if constexpr (CW == 2) {
    const float2 x = 0 < n ? *reinterpret_cast<const float2 *>(p) : make_float2(0.f, 0.f);
    v[0] = x.x; v[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < CW / 4; ++i) {
      const float4 x = 4 * i < n ? *reinterpret_cast<const float4 *>(p + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
      v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
    }
  }
}
template <int CW>
__device__ __forceinline__ void store_cols_f32(float *p, const float (&v)[CW], int n, bool aligned) {
  if (!aligned) {
#pragma unroll
    for (int c = 0; c < CW; ++c)
      if (c < n) p[c] = v[c];
  } else if constexpr (CW == 2) {
    if (0 < n) *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
  } else {
#pragma unroll
    for (int i = 0; i < CW / 4; ++i)
      if (4 * i < n) *reinterpret_cast<float4 *>(p + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

constexpr int kMaxWarps = 8, kMaxStages = 3;

// Values of a stage: what a kind needs of the two records.
__host__ __device__ constexpr int stage_keys(int NP, What what) { return (what == kSave ? 2 : 3) * kC * NP; }
__host__ __device__ constexpr int stage_heads(What what) { return (what == kSave ? 1 : 2) * kTri + kScal; }
__host__ __device__ constexpr int stage_values(int NP, What what) { return stage_keys(NP, what) + stage_heads(what); }

// One sequence of one head, columns p0 = CW * (group * warps + warp) ... OWN: the copies have a warp of their own.
template <int J, int CW, What WHAT, bool OWN>
__device__ __forceinline__ void run(const DeltaArgs &a, int group, int warps, int stages, bool aligned) {
  constexpr int NP = 32 * J, kStage = stage_values(NP, WHAT);
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem);  // full and free of each stage
  float *stage0 = reinterpret_cast<float *>(smem + 128);
  const int64_t h = blockIdx.y, b = blockIdx.z, bh = b * a.H + h, hk = h / (a.H / a.Hk);
  const int64_t len = live_steps(a.lengths, b, a.L), chunks = (len + kC - 1) / kC;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&bars[s], 1);
      mbar_init(&bars[kMaxStages + s], warps);
    }
    mbar_fence_init();
  }
  __syncthreads();

  // A lane copies the records of chunk i (of the order they are gone through) into their stage. Every wait of a
  // role on another is bounded: when one has run out, anywhere in the launch, the lane asks for nothing more and
  // each warp leaves its chunks at its next unfinished wait, so that nothing works on records that are not there.
  const float *keys = a.keys + (b * a.Hk + hk) * a.nC * key_values(NP);
  const float *heads = a.heads + bh * a.nC * head_values(WHAT != kForward) + (WHAT == kBack ? kTri : 0);
  int64_t asked = 0;  // chunks whose records the lane has asked for
  bool going = true;
  const auto refill = [&](int64_t i, int s, int turn) {
    const int64_t chunk = WHAT == kBack ? chunks - 1 - i : i;
    // all warps are done with the stage, hence its copies have landed
    going = going && (!turn || wait_bar(&bars[kMaxStages + s], (turn - 1) & 1, a.err, a.wait_ns));
    if (!going) return;
    float *st = stage0 + s * kStage;
    mbar_expect_tx(&bars[s], 4 * kStage);
    bulk_load(st, keys + chunk * key_values(NP), 4 * stage_keys(NP, WHAT), &bars[s]);
    bulk_load(st + stage_keys(NP, WHAT), heads + chunk * head_values(WHAT != kForward), 4 * stage_heads(WHAT), &bars[s]);
    ++asked;
  };
  const auto drain = [&]() {  // the last copies into each stage have landed
    for (int64_t i = max(asked - stages, (int64_t)0); i < asked; ++i) wait_own(&bars[i % stages], (i / stages) & 1, a.err);
  };
  const bool copies = warp == (OWN ? warps : 0) && lane == 0;
  // a short limit runs out here: nothing has been asked for yet
  if (copies && chunks > 0 && a.wait_ns < kShortNs) going = wait_slow<false>(&bars[0], 0, a.err, a.wait_ns);
  if (OWN && warp == warps) {
    if (!copies) return;
    int s = 0, turn = 0;
    for (int64_t i = 0; i < chunks && going; ++i) {
      refill(i, s, turn);
      if (++s == stages) s = 0, ++turn;
    }
    drain();
    return;
  }
  if (!OWN && copies)
    for (int i = 0; i < min((int64_t)(stages - 1), chunks); ++i) refill(i, i, 0);

  float *hs = stage0 + stages * kStage + warp * Warp<CW>::values(NP, WHAT);  // the state's values
  float *b0 = hs + (NP / 2) * Warp<CW>::LD, *b1 = b0 + (kC / 2) * Warp<CW>::LD;
  const int p0 = CW * (group * warps + warp);
  const int N = (int)a.N, n_in = min(CW, (int)a.P - p0), n_room = min(CW, (int)a.Pp - p0);
  // a warp without columns goes along with nothing to load or store
  const float *from = WHAT == kBack ? a.dh_final : a.h0;
  float st[J][CW];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int n = 32 * j + lane;
    const bool on = from != nullptr && n < N;
    load_cols_f32<CW>(st[j], on ? from + (bh * N + n) * a.P + p0 : nullptr, on ? n_in : 0, aligned);
  }
  // v (dy) of the lane's step in a chunk, loaded a chunk ahead
  const float *in = static_cast<const float *>(WHAT == kBack ? a.dy : a.v) + (b * a.L * a.H + h) * a.P + p0;
  const int64_t step = a.H * a.P;
  float nx[CW];
  const auto fetch = [&](int64_t chunk) {
    const int64_t t = chunk * kC + lane;
    load_cols_f32<CW>(nx, in + (t < len ? t : 0) * step, t < len ? n_in : 0, aligned);
  };
  if (chunks > 0) fetch(WHAT == kBack ? chunks - 1 : 0);
  int s = 0, turn = 0;
  for (int64_t i = 0; i < chunks; ++i) {
    // without a warp for the copies: into the stage of the chunk before, which the other warps are done
    // with in a moment
    if (!OWN && copies && i + stages - 1 < chunks) refill(i + stages - 1, s ? s - 1 : stages - 1, s ? turn + 1 : turn);
    const int64_t chunk = WHAT == kBack ? chunks - 1 - i : i, t = chunk * kC + lane;
    const float *key = stage0 + s * kStage, *head = key + stage_keys(NP, WHAT);
    const float4 *K = reinterpret_cast<const float4 *>(key) + lane, *KT = reinterpret_cast<const float4 *>(key + kC * NP) + lane,
                 *third = reinterpret_cast<const float4 *>(key + 2 * kC * NP) + lane;
    const float *scal = head + (WHAT == kBack ? 0 : kTri);
    float v[CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) v[c] = nx[c];
    if (i + 1 < chunks) fetch(WHAT == kBack ? chunk - 1 : chunk + 1);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int n = 32 * j + lane;
      put<CW>(hs, n, st[j]);
      if (WHAT == kSave && n < N) store_cols_f32<CW>(a.carry + ((bh * a.nC + chunk) * N + n) * a.Pp + p0, st[j], n_room, true);
      if (WHAT == kBack && n < N) store_cols_f32<CW>(a.xcarry + ((bh * a.nC + chunk) * N + n) * a.Pp + p0, st[j], n_room, true);
    }
    __syncwarp();
    if (!__all_sync(0xffffffffu, wait_bar(&bars[s], turn & 1, a.err, a.wait_ns))) break;
    const float grow = scal[lane], fade = scal[kC + lane], beta = scal[2 * kC + lane], last = scal[3 * kC], rest = scal[3 * kC + 1];
    if constexpr (WHAT != kBack) {
      float y[CW];
      {
        pair2 acc[CW] = {};
        mul<CW, NP / 4>(K, 32, hs, acc);
#pragma unroll
        for (int c = 0; c < CW; ++c) v[c] = fmaf(-grow, both(acc[c]), v[c]);
      }
      put<CW>(b0, lane, v);
      __syncwarp();
      {
        pair2 acc[CW] = {};
        mul<CW, kC / 4>(reinterpret_cast<const float4 *>(head) + lane, 32, b0, acc);
#pragma unroll
        for (int c = 0; c < CW; ++c) v[c] = both(acc[c]);
      }
      if (WHAT == kSave && t < len) store_cols_f32<CW>(a.e + (bh * a.L + t) * a.Pp + p0, v, n_room, true);
      if constexpr (WHAT == kForward) {
        pair2 acc[CW] = {};
        mul<CW, NP / 4>(third, 32, hs, acc);
#pragma unroll
        for (int c = 0; c < CW; ++c) y[c] = a.scale * grow * both(acc[c]);
      }
#pragma unroll
      for (int c = 0; c < CW; ++c) v[c] *= beta;
      if (WHAT == kForward) put<CW>(b1 + (kC / 2) * Warp<CW>::LD, lane, v);
#pragma unroll
      for (int c = 0; c < CW; ++c) v[c] *= fade;
      put<CW>(b1, lane, v);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < J; ++j) {
        pair2 acc[CW] = {};
        mul<CW, kC / 4>(KT + 32 * j, NP, b1, acc);
#pragma unroll
        for (int c = 0; c < CW; ++c) st[j][c] = fmaf(last, st[j][c], fmaf(rest, st[j][c], both(acc[c])));
      }
      if constexpr (WHAT == kForward) {
        pair2 acc[CW] = {};
        mul<CW, kC / 4>(reinterpret_cast<const float4 *>(head + kTri + kScal) + lane, 32, b1 + (kC / 2) * Warp<CW>::LD, acc);
#pragma unroll
        for (int c = 0; c < CW; ++c) y[c] += both(acc[c]);
        if (t < len) store_cols_f32<CW>(static_cast<float *>(a.y) + (b * a.L * a.H + h) * a.P + p0 + t * step, y, n_in, aligned);
      }
    } else {
      float *b2 = b1 + (kC / 2) * Warp<CW>::LD, *b3 = b2 + (kC / 2) * Warp<CW>::LD;
      float w[CW];
      put<CW>(b0, lane, v);
#pragma unroll
      for (int c = 0; c < CW; ++c) w[c] = a.scale * grow * v[c];
      put<CW>(b1, lane, w);
      __syncwarp();
      {
        pair2 acc[CW] = {};
        mul<CW, kC / 4>(reinterpret_cast<const float4 *>(head + kScal + kTri) + lane, 32, b0, acc);
#pragma unroll
        for (int c = 0; c < CW; ++c) w[c] = both(acc[c]);
      }
      {
        pair2 acc[CW] = {};
        mul<CW, NP / 4>(K, 32, hs, acc);
#pragma unroll
        for (int c = 0; c < CW; ++c) w[c] = fmaf(fade, both(acc[c]), w[c]);
      }
      put<CW>(b2, lane, w);
      __syncwarp();
      {
        pair2 acc[CW] = {};
        mul<CW, kC / 4>(reinterpret_cast<const float4 *>(head + kScal) + lane, 32, b2, acc);
#pragma unroll
        for (int c = 0; c < CW; ++c) w[c] = both(acc[c]);
      }
      if (t < len) store_cols_f32<CW>(a.du + (bh * a.L + t) * a.Pp + p0, w, n_room, true);
#pragma unroll
      for (int c = 0; c < CW; ++c) w[c] *= beta;
      if (t < len) store_cols_f32<CW>(static_cast<float *>(a.dv) + (b * a.L * a.H + h) * a.P + p0 + t * step, w, n_in, aligned);
#pragma unroll
      for (int c = 0; c < CW; ++c) w[c] *= -grow;
      put<CW>(b3, lane, w);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < J; ++j) {
        pair2 acc[CW] = {};
        mul<CW, kC / 4>(third + 32 * j, NP, b1, acc);
        mul<CW, kC / 4>(KT + 32 * j, NP, b3, acc);
#pragma unroll
        for (int c = 0; c < CW; ++c) st[j][c] = fmaf(last, st[j][c], fmaf(rest, st[j][c], both(acc[c])));
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[kMaxStages + s]);
    if (++s == stages) s = 0, ++turn;
  }
  if (!OWN && copies) drain();
  if (WHAT != kSave) {
    float *out = WHAT == kBack ? a.dh0 : a.h_final;
    const bool bad = len > 0 && __any_sync(0xffffffffu, timed_out(a.err));
    if (bad) {
      __syncwarp();
      fill_nan(WHAT == kBack ? a.dv : a.y, false, (b * a.L * a.H + h) * a.P + p0, len, step, n_in, lane, 32);
      fill_nan(out, false, bh * N * a.P + p0, N, a.P, n_in, lane, 32);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int n = 32 * j + lane;
      if (out && n < N && !bad) store_cols_f32<CW>(out + (bh * N + n) * a.P + p0, st[j], n_in, aligned);
    }
    const float zero[CW] = {};
    float *rows = static_cast<float *>(WHAT == kBack ? a.dv : a.y) + (b * a.L * a.H + h) * a.P + p0;
    for (int64_t t = len + lane; t < a.L; t += 32) store_cols_f32<CW>(rows + t * step, zero, n_in, aligned);
  }
}

template <int J, int CW, bool OWN>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) delta_rows_kernel(DeltaArgs a, int warps, int stages, bool aligned) {
  run<J, CW, kForward, OWN>(a, blockIdx.x, warps, stages, aligned);
}

// The states and the adjoints of a backward pass do not need one another: their blocks take turns.
template <int J, int CW, bool OWN>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) delta_rows_both_kernel(DeltaArgs a, int warps, int stages, bool aligned) {
  if (blockIdx.x & 1) run<J, CW, kBack, OWN>(a, blockIdx.x >> 1, warps, stages, aligned);
  else run<J, CW, kSave, OWN>(a, blockIdx.x >> 1, warps, stages, aligned);
}

template <int J, int CW>
cudaError_t launch_jc(const DeltaArgs &a, bool bwd, const char *name, cudaStream_t st) {
  constexpr int NP = 32 * J;
  const int all = (int)((a.Pp + CW - 1) / CW);  // the padded columns of the workspace rows are written too
  // the warps of a block share its records: as few as give one block an SM, or eight
  const int64_t slices = a.Bt * a.H * (bwd ? 2 : 1);
  int warps = 1;
  while (warps < kMaxWarps && slices * ((all + warps - 1) / warps) > 148) ++warps;
  warps = std::min(warps, all);
  const auto bytes = [&](int stages) {
    const int f = 4 * (stages * stage_values(NP, kForward) + warps * Warp<CW>::values(NP, kForward));
    const int s = 4 * (stages * stage_values(NP, kSave) + warps * Warp<CW>::values(NP, kSave));
    const int k = 4 * (stages * stage_values(NP, kBack) + warps * Warp<CW>::values(NP, kBack));
    return 128 + (bwd ? std::max(s, k) : f);
  };
  const int stages = bytes(kMaxStages) <= 227 * 1024 ? kMaxStages : 2, smem = bytes(stages);
  const bool own = warps < kMaxWarps;
  auto kern = bwd ? (own ? delta_rows_both_kernel<J, CW, true> : delta_rows_both_kernel<J, CW, false>)
                  : (own ? delta_rows_kernel<J, CW, true> : delta_rows_kernel<J, CW, false>);
  cudaError_t e = allow_shared(kern);
  if (e != cudaSuccess || (e = trace_before(st, name)) != cudaSuccess) return e;
  uintptr_t all16 = reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(bwd ? a.dy : a.y);
  all16 |= reinterpret_cast<uintptr_t>(a.h0) | reinterpret_cast<uintptr_t>(a.h_final) | reinterpret_cast<uintptr_t>(a.dv) |
           reinterpret_cast<uintptr_t>(a.dh_final) | reinterpret_cast<uintptr_t>(a.dh0);
  const dim3 grid((unsigned)((all + warps - 1) / warps) * (bwd ? 2 : 1), (unsigned)a.H, (unsigned)a.Bt);
  kern<<<grid, 32 * (warps + own), smem, st>>>(a, warps, stages, a.P % 4 == 0 && all16 % 16 == 0);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : trace_after(st);
}

template <int J>
cudaError_t launch_j(const DeltaArgs &a, bool bwd, cudaStream_t st) {
  constexpr int smem = 4 * kPrepWarps * prep_values<32 * J>();
  auto prep = bwd ? delta_rows_prep_kernel<32 * J, true> : delta_rows_prep_kernel<32 * J, false>;
  cudaError_t e = cudaFuncSetAttribute(prep, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess || (e = trace_before(st, "delta_rows_prep")) != cudaSuccess) return e;
  prep<<<dim3((unsigned)((a.nC + kPrepWarps - 1) / kPrepWarps), (unsigned)a.Hk, (unsigned)a.Bt), 32 * kPrepWarps, smem, st>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || (e = trace_after(st)) != cudaSuccess) return e;
  const char *name = bwd ? "delta_rows_both" : "delta_rows";
  // eight columns a warp read less for each FMA; four or two make more warps where there are few
  // (32 sequences of 18,000 steps, 32 x 32, without a warp for the copies: 703 us with four, 652 with two)
  const int64_t of4 = a.Bt * a.H * ((a.P + 3) / 4) * (bwd ? 2 : 1);
  if (of4 <= 2 * 148) return launch_jc<J, 2>(a, bwd, name, st);
  if (of4 <= 8 * 148) return launch_jc<J, 4>(a, bwd, name, st);
  return launch_jc<J, 8>(a, bwd, name, st);
}

}  // namespace

int64_t delta_rows_key_bytes(int64_t N) { return 4 * (int64_t)key_values(N <= 32 ? 32 : N <= 64 ? 64 : 128); }
int64_t delta_rows_head_bytes(bool bwd) { return 4 * (int64_t)head_values(bwd); }

cudaError_t launch_delta_rows(const DeltaArgs &a, bool bwd, cudaStream_t st) {
  if (a.C != kC) return cudaErrorInvalidValue;
  return a.N <= 32 ? launch_j<1>(a, bwd, st) : a.N <= 64 ? launch_j<2>(a, bwd, st) : launch_j<4>(a, bwd, st);
}

}  // namespace pdssm
