// Gradients of queries, keys, decays and betas of the gated delta rule, chunk by chunk in
// parallel (bf16 inputs), from what the chunked passes wrote: the states H at the chunks'
// ends, the adjoints X there, e, du and <dy, y> in fp32 (csrc/delta_chunk.cu, delta_chunk_bwd.cuh).
//
// With D_ij = exp(G_i - G_j), u = beta e, and for the chunk's rows
//   F1_ij = scale D_ij <dy_i, u_j> (j <= i),   F2_ij = -beta_i D_ij <du_i, u_j> (j < i):
//   dq = scale diag(exp G) dY H^T + F1 K
//   dk = diag(fade) U X^T - diag(beta exp G) dU H^T + F1^T Q + (F2 + F2^T) K,  fade = exp(G_64 - G)
//   dbeta_i = <du_i, e_i>
//   dg_i = <X, H'> + sum over j >= i of (<dy_j, y_j> - beta_j <du_j, v_j>)
// (X and H' at the chunk's end). The last line is the scaling identity of the recurrence:
// making every state from step i on larger by a factor scales the outputs, and what the
// values contribute does not take part. It needs no product but three dot products a row,
// which stay in fp32, so dg is exact to fp32's rounding of the sum's terms: off by some 2^-24 of
// |<X, H'>| + sum over j >= i of (|<dy_j, y_j>| + beta_j |<du_j, v_j>|). Its value has the factor
// exp(g_i), which no single term has: where the decay is strong, that is rounding of terms that cancel,
// not of dg (csrc/delta_grad.cu sums terms that have the factor). Where exp(g_i) is 0 in fp32 dg_i is 0.
//
// The products have 64 rows (steps) and run on the tensor cores, operands in shared memory as two
// bf16 parts (16 bits; dq and dk are rounded to bf16). Row scalings are applied where an
// accumulator is read, so each operand is stored once. The value heads that share a key
// head are gone through in the block; their sum stays in registers.
// What bounds it: the alternation of loads and products in a block (one block an SM for
// N = P = 128, two for 64), then HBM (e, du and the two states are fp32): 256 sequences of 2,048 steps,
// 64 x 64: 330 us, 128 of 4,096 steps, 128 x 128: 790 us; the bytes alone would take about 165 and 370.
#include <algorithm>

#include "delta.cuh"
#include "delta_chunk.cuh"
#include "sm100.cuh"

namespace pdssm {

using namespace sm100;

namespace {

constexpr int kThreads = 512;  // 16 warps: the loads of a phase are what it waits for

template <int NP, int PP>
struct Layout {
  static constexpr int kKq = (NP / 8) * kChunkGroup, kRow = (PP / 8) * kChunkGroup;  // K or Q; a rows-by-p part
  static constexpr int kHGroup = NP * 16 + 16, kH = (PP / 8) * kHGroup;              // a part of H or X
  static constexpr int kYo = 2 * kKq, kDo = kYo + kRow, kUo = kDo + 2 * kRow, kHo = kUo + 2 * kRow, kFo = kHo + 2 * kH;
  static constexpr int kScal = kFo + 4 * kSquare;                 // the record's scalars
  static constexpr int kRed = kScal + kScalars;                   // dG, dbeta (64 floats each), <X, H'> by warp
  static constexpr int kBar = kRed + 4 * (2 * kChunk + 16), kBytes = kBar + 24;
  // tensor memory: the two squares; dY H^T, then F1 K; dU H^T, then the other products of dk;
  // U X^T, for N <= 64 in the place of the squares
  static constexpr int kP1 = 0, kP2 = 64, kI1 = 128, kI2 = 128 + NP, kUx = NP == 64 ? 0 : 128 + 2 * NP, kCols = NP == 64 ? 256 : 512;
  static constexpr int WN = NP / 8;  // a thread's columns of an accumulator of NP
};

__device__ __forceinline__ float sum4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

// Eight values as two bf16 parts.
__device__ __forceinline__ void put_parts(uint8_t *hi, uint8_t *lo, float4 a, float4 b) {
  uint32_t p[2][4];
  split2(a.x, a.y, p[0][0], p[1][0]);
  split2(a.z, a.w, p[0][1], p[1][1]);
  split2(b.x, b.y, p[0][2], p[1][2]);
  split2(b.z, b.w, p[0][3], p[1][3]);
  *reinterpret_cast<uint4 *>(hi) = make_uint4(p[0][0], p[0][1], p[0][2], p[0][3]);
  *reinterpret_cast<uint4 *>(lo) = make_uint4(p[1][0], p[1][1], p[1][2], p[1][3]);
}

__device__ __forceinline__ float4 times(float4 a, float s) { return make_float4(a.x * s, a.y * s, a.z * s, a.w * s); }
__device__ __forceinline__ float4 low4(uint4 v) { return make_float4(low_half(v.x), high_half(v.x), low_half(v.y), high_half(v.y)); }
__device__ __forceinline__ float4 high4(uint4 v) { return make_float4(low_half(v.z), high_half(v.z), low_half(v.w), high_half(v.w)); }

template <int NP, int PP>
__global__ void __launch_bounds__(kThreads, NP == 64 && PP == 64 ? 2 : 1) delta_chunk_grad_kernel(DeltaArgs a, bool wide, bool wide_v, bool wide_out) {
  using Lay = Layout<NP, PP>;
  constexpr int WN = Lay::WN, PG = PP / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  float *scal = reinterpret_cast<float *>(smem + Lay::kScal), *sdG = reinterpret_cast<float *>(smem + Lay::kRed), *sdb = sdG + kChunk,
        *sxh = sdb + kChunk;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::kBar);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 2), *bad = tslot + 1;  // bad: a wait of the call has run out
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int64_t chunk = blockIdx.x, hk = blockIdx.y, b = blockIdx.z, t0 = chunk * kChunk;
  const int64_t len = live_steps(a.lengths, b, a.L), row0 = b * a.L + t0;
  const int rows = (int)min((int64_t)kChunk, a.L - t0), live = (int)max((int64_t)0, min((int64_t)kChunk, len - t0));
  const int r_heads = (int)(a.H / a.Hk), N = (int)a.N, P = (int)a.P, Pp = (int)a.Pp;
  const bool gb = a.gate_t == PDSSM_BF16;
  using B = __nv_bfloat16;
  if (live == 0) {
    for (int i = tid; i < rows * N; i += kThreads) {
      const int64_t at = ((row0 + i / N) * a.Hk + hk) * N + i % N;
      static_cast<B *>(a.dq)[at] = __float2bfloat16_rn(0.f);
      static_cast<B *>(a.dk)[at] = __float2bfloat16_rn(0.f);
    }
    for (int i = tid; i < rows * r_heads; i += kThreads) {
      const int64_t at = (row0 + i / r_heads) * a.H + hk * r_heads + i % r_heads;
      store_any(a.dg, at, gb, 0.f);
      store_any(a.dbeta, at, gb, 0.f);
    }
    return;
  }
  if (tid == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    mbar_fence_init();
    *bad = timed_out(a.err);
  }
  if (warp == 0) {
    tmem_alloc(tslot, Lay::kCols);
    tmem_relinquish();
  }
  load_tile<NP / 8, kChunkGroup, 16, kThreads>(smem, static_cast<const B *>(a.k), row0, a.Hk, hk, a.N, 0, live, wide, tid);
  load_tile<NP / 8, kChunkGroup, 16, kThreads>(smem + Lay::kKq, static_cast<const B *>(a.q), row0, a.Hk, hk, a.N, 0, live, wide, tid);
  cp_async_commit();
  const uint32_t sbase = smem_u32(smem);
  uint32_t tbase = 0, tq = 0;
  const bool whole = N == NP && Pp == PP && P == PP && wide_v;

  // the thread's row of an accumulator and its part of the columns
  const int quarter = warp & 3, row = 16 * quarter + (lane & 15), up = warp >> 2, part = 2 * up + (lane >> 4);
  float dq[WN] = {}, dk[WN] = {};

  for (int hh = 0; hh < r_heads; ++hh) {
    const int64_t h = hk * r_heads + hh, bh = b * a.H + h;
    const uint32_t ph = hh & 1;
    const float *carry = a.carry + (bh * (a.nC + 1) + chunk) * a.N * a.Pp;
    const float *xcarry = a.xcarry + (bh * a.nC + chunk) * a.N * a.Pp;
    // What the first products need is asked for ahead of its use. A whole chunk of whole rows is loaded
    // without conditions: a branch around each load makes them wait for one another.
    constexpr int kRows = kChunk * PG / kThreads, kPer = NP * PG / kThreads;
    const int g = tid % PG, r0 = tid / PG;
    constexpr int kEvery = kThreads / PG;  // a thread's rows are kEvery apart
    const float *rec = reinterpret_cast<const float *>(a.records + (bh * a.nC + chunk) * a.rec_bytes + a.rec_bytes - kScalars);
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 e[kRows][2], du[kRows][2], yy[kRows], sx[kPer][2];
    uint4 dy[kRows], v[kRows];
    float beta[kRows];
    const auto fetch_rows = [&](bool all) {
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int c = r0 + k * kEvery;
        const bool on = all || c < live;
        const int64_t row = bh * a.L + t0 + c, at = ((row0 + c) * a.H + h) * P + 8 * g;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bool here = all || (on && 8 * g + 4 * s < Pp);
          e[k][s] = here ? *reinterpret_cast<const float4 *>(a.e + row * Pp + 8 * g + 4 * s) : none;
          du[k][s] = here ? *reinterpret_cast<const float4 *>(a.du + row * Pp + 8 * g + 4 * s) : none;
        }
        yy[k] = on ? *reinterpret_cast<const float4 *>(a.dyy + row * 4) : none;
        if (all || (wide_v && on && 8 * g < P)) {
          dy[k] = *reinterpret_cast<const uint4 *>(static_cast<const B *>(a.dy) + at);
          v[k] = *reinterpret_cast<const uint4 *>(static_cast<const B *>(a.v) + at);
        } else {
          dy[k] = gather8(static_cast<const B *>(a.dy) + at, on && !wide_v ? P - 8 * g : 0);
          v[k] = gather8(static_cast<const B *>(a.v) + at, on && !wide_v ? P - 8 * g : 0);
        }
        beta[k] = rec[2 * kChunk + c];
      }
    };
    // a state of the workspace into registers, and from there as operands
    const auto fetch_state = [&](const float *from, float4 (&x)[kPer][2]) {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int n = r0 + k * kEvery;
          if (whole) x[k][s] = *reinterpret_cast<const float4 *>(from + n * PP + 8 * g + 4 * s);
          else x[k][s] = n < N && 8 * g + 4 * s < Pp ? *reinterpret_cast<const float4 *>(from + n * Pp + 8 * g + 4 * s) : none;
        }
    };
    const auto put_state = [&](const float4 (&x)[kPer][2]) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        uint8_t *to = smem + Lay::kHo + g * Lay::kHGroup + (r0 + k * kEvery) * 16;
        put_parts(to, to + Lay::kH, x[k][0], x[k][1]);
      }
    };
    if (whole && live == kChunk) fetch_rows(true);
    else fetch_rows(false);
    if (kRows == 1) fetch_state(carry, sx);
    if (tid < kScalars / 16) reinterpret_cast<float4 *>(scal)[tid] = reinterpret_cast<const float4 *>(rec)[tid];
    // rows: dy, du, u as operands, and the dot products of the gates' gradients
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int c = r0 + k * kEvery;
      float db = sum4(du[k][0], e[k][0], sum4(du[k][1], e[k][1], 0.f));
      float dG = -beta[k] * sum4(low4(v[k]), du[k][0], sum4(high4(v[k]), du[k][1], 0.f));
#pragma unroll
      for (int o = PG / 2; o > 0; o >>= 1) {
        db += __shfl_xor_sync(0xffffffffu, db, o);
        dG += __shfl_xor_sync(0xffffffffu, dG, o);
      }
      if (g == 0) {
        sdb[c] = db;
        sdG[c] = dG + ((yy[k].x + yy[k].y) + (yy[k].z + yy[k].w));
      }
      const int off = g * kChunkGroup + c * 16;
      *reinterpret_cast<uint4 *>(smem + Lay::kYo + off) = dy[k];
      put_parts(smem + Lay::kDo + off, smem + Lay::kDo + Lay::kRow + off, du[k][0], du[k][1]);
      put_parts(smem + Lay::kUo + off, smem + Lay::kUo + Lay::kRow + off, times(e[k][0], beta[k]), times(e[k][1], beta[k]));
    }
    if (kRows != 1) fetch_state(carry, sx);
    put_state(sx);
    cp_async_wait<0>();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (hh == 0) {
      tbase = __shfl_sync(0xffffffffu, *tslot, 0);
      tq = tbase + ((uint32_t)(32 * quarter) << 16);
    }
    constexpr uint32_t idS = idesc_bf16_f32(64, kChunk, false, false), idN = idesc_bf16_f32(64, NP, false, false);
    if (warp == 0) {
      if (elect_one()) {
        const uint64_t y = smem_desc(sbase + Lay::kYo, kChunkGroup, 128), d = smem_desc(sbase + Lay::kDo, kChunkGroup, 128),
                       u = smem_desc(sbase + Lay::kUo, kChunkGroup, 128), m = smem_desc(sbase + Lay::kHo, Lay::kHGroup, 128);
        constexpr uint32_t R = Lay::kRow >> 4, Hp = Lay::kH >> 4;
#pragma unroll
        for (int ks = 0; ks < PP / 16; ++ks) {
          const uint32_t o = 2 * kChunkGroup * ks >> 4, oh = 2 * Lay::kHGroup * ks >> 4;
          mma_bf16(tbase + Lay::kP1, y + o, u + o, idS, ks > 0);
          mma_bf16(tbase + Lay::kP1, y + o, u + R + o, idS, 1);
          mma_bf16(tbase + Lay::kP2, d + o, u + o, idS, ks > 0);
          mma_bf16(tbase + Lay::kP2, d + o, u + R + o, idS, 1);
          mma_bf16(tbase + Lay::kP2, d + R + o, u + o, idS, 1);
          mma_bf16(tbase + Lay::kI1, y + o, m + oh, idN, ks > 0);
          mma_bf16(tbase + Lay::kI1, y + o, m + Hp + oh, idN, 1);
          mma_bf16(tbase + Lay::kI2, d + o, m + oh, idN, ks > 0);
          mma_bf16(tbase + Lay::kI2, d + o, m + Hp + oh, idN, 1);
          mma_bf16(tbase + Lay::kI2, d + R + o, m + oh, idN, 1);
        }
        mma_commit(&bars[0]);
      }
      __syncwarp();
    }
    // X, and its product with the state behind the chunk, while the tensor core works
    float xh = 0.f;
    {
      float4 sh[kPer][2];
      fetch_state(xcarry, sx);
      fetch_state(carry + a.N * a.Pp, sh);
#pragma unroll
      for (int k = 0; k < kPer; ++k) xh = sum4(sx[k][0], sh[k][0], sum4(sx[k][1], sh[k][1], xh));
    }
    if (!wait_own(&bars[0], ph, a.err)) *bad = 1;
    tc_fence_after();
    put_state(sx);
    {
      const float hi = scal[4 * kChunk + row], lo = scal[5 * kChunk + row], beta = scal[2 * kChunk + row];
      float p1[8], p2[8];
      load_cols<64, 8>(tq + Lay::kP1 + 16 * up, p1);
      load_cols<64, 8>(tq + Lay::kP2 + 16 * up, p2);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int j = 8 * part + s;
        const float D = decay2((hi - scal[4 * kChunk + j]) + (lo - scal[5 * kChunk + j]));
        p1[s] = j <= row ? a.scale * D * p1[s] : 0.f;
        p2[s] = j < row ? -beta * D * p2[s] : 0.f;
      }
      uint8_t *to = smem + Lay::kFo + part * 1024 + row * 16;
      put_parts(to, to + kSquare, make_float4(p1[0], p1[1], p1[2], p1[3]), make_float4(p1[4], p1[5], p1[6], p1[7]));
      put_parts(to + 2 * kSquare, to + 3 * kSquare, make_float4(p2[0], p2[1], p2[2], p2[3]), make_float4(p2[4], p2[5], p2[6], p2[7]));
      const float fq = a.scale * scal[row], fk = -beta * scal[row];
      float t[WN];
      load_cols<64, WN>(tq + Lay::kI1 + 2 * WN * up, t);
#pragma unroll
      for (int n = 0; n < WN; ++n) dq[n] = fmaf(fq, t[n], dq[n]);
      load_cols<64, WN>(tq + Lay::kI2 + 2 * WN * up, t);
#pragma unroll
      for (int n = 0; n < WN; ++n) dk[n] = fmaf(fk, t[n], dk[n]);
    }
    {
      float s = xh;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) sxh[warp] = s;
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) {
      if (elect_one()) {
        constexpr uint32_t idF = idesc_bf16_f32(64, NP, false, true), idFt = idesc_bf16_f32(64, NP, true, true);
        const uint64_t u = smem_desc(sbase + Lay::kUo, kChunkGroup, 128), m = smem_desc(sbase + Lay::kHo, Lay::kHGroup, 128),
                       f = smem_desc(sbase + Lay::kFo, 1024, 128), ft = smem_desc(sbase + Lay::kFo, 128, 1024),
                       kt = smem_desc(sbase, 128, kChunkGroup), qt = smem_desc(sbase + Lay::kKq, 128, kChunkGroup);
        constexpr uint32_t R = Lay::kRow >> 4, Hp = Lay::kH >> 4, S = kSquare >> 4;
#pragma unroll
        for (int ks = 0; ks < PP / 16; ++ks) {
          const uint32_t o = 2 * kChunkGroup * ks >> 4, oh = 2 * Lay::kHGroup * ks >> 4;
          mma_bf16(tbase + Lay::kUx, u + o, m + oh, idN, ks > 0);
          mma_bf16(tbase + Lay::kUx, u + o, m + Hp + oh, idN, 1);
          mma_bf16(tbase + Lay::kUx, u + R + o, m + oh, idN, 1);
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t of = 2048 * ks >> 4, ot = 256 * ks >> 4;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            mma_bf16(tbase + Lay::kI1, f + q * S + of, kt + ot, idF, ks + q > 0);
            mma_bf16(tbase + Lay::kI2, ft + q * S + ot, qt + ot, idFt, ks + q > 0);
            mma_bf16(tbase + Lay::kI2, f + (2 + q) * S + of, kt + ot, idF, 1);
            mma_bf16(tbase + Lay::kI2, ft + (2 + q) * S + ot, kt + ot, idFt, 1);
          }
        }
        mma_commit(&bars[1]);
      }
      __syncwarp();
    }
    if (warp == 1) {
      // dg: what reaches the chunk's end reaches every step of it; two steps a lane
      double s = (double)sdG[2 * lane] + (double)sdG[2 * lane + 1], end = 0;
#pragma unroll
      for (int w = 0; w < 16; ++w) end += sxh[w];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double dn = __shfl_down_sync(0xffffffffu, s, o);
        if (lane + o < 32) s += dn;
      }
      s += end;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int c = 2 * lane + k;
        if (c < rows) {
          const int64_t at = (row0 + c) * a.H + h;
          // the gate to the base 2 from its running sum; exp2(-150) is 0
          const float *hi = scal + 4 * kChunk + c, *lo = scal + 5 * kChunk + c;
          const float g2 = c ? (hi[0] - hi[-1]) + (lo[0] - lo[-1]) : hi[0] + lo[0];
          store_any(a.dg, at, gb, c < live && !(g2 <= -150.f) ? (float)(k ? s - (double)sdG[2 * lane] : s) : 0.f);
          store_any(a.dbeta, at, gb, c < live ? sdb[c] : 0.f);
        }
      }
    }
    if (!wait_own(&bars[1], ph, a.err)) *bad = 1;
    tc_fence_after();
    {
      const float fade = scal[kChunk + row];
      float t[WN];
      load_cols<64, WN>(tq + Lay::kUx + 2 * WN * up, t);
#pragma unroll
      for (int n = 0; n < WN; ++n) dk[n] = fmaf(fade, t[n], dk[n]);
      load_cols<64, WN>(tq + Lay::kI1 + 2 * WN * up, t);
#pragma unroll
      for (int n = 0; n < WN; ++n) dq[n] += t[n];
      load_cols<64, WN>(tq + Lay::kI2 + 2 * WN * up, t);
#pragma unroll
      for (int n = 0; n < WN; ++n) dk[n] += t[n];
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (row < rows) {
    const int n0 = part * WN;
    const int64_t at = ((row0 + row) * a.Hk + hk) * N + n0;
    B *oq = static_cast<B *>(a.dq) + at, *ok = static_cast<B *>(a.dk) + at;
    const bool on = row < live;
#pragma unroll
    for (int n = 0; n < WN; n += 8) {
      if (wide_out) {
        if (n0 + n < N) {
          uint32_t q[4], k[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            q[s] = on ? pack_bf16(dq[n + 2 * s], dq[n + 2 * s + 1]) : 0;
            k[s] = on ? pack_bf16(dk[n + 2 * s], dk[n + 2 * s + 1]) : 0;
          }
          *reinterpret_cast<uint4 *>(oq + n) = make_uint4(q[0], q[1], q[2], q[3]);
          *reinterpret_cast<uint4 *>(ok + n) = make_uint4(k[0], k[1], k[2], k[3]);
        }
      } else {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          if (n0 + n + s < N) {
            oq[n + s] = __float2bfloat16_rn(on ? dq[n + s] : 0.f);
            ok[n + s] = __float2bfloat16_rn(on ? dk[n + s] : 0.f);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tbase, Lay::kCols);
  if (*bad) {
    fill_nan(a.dq, true, (row0 * a.Hk + hk) * N, live, a.Hk * N, N, tid, kThreads);
    fill_nan(a.dk, true, (row0 * a.Hk + hk) * N, live, a.Hk * N, N, tid, kThreads);
    fill_nan(a.dg, gb, row0 * a.H + hk * r_heads, live, a.H, r_heads, tid, kThreads);
    fill_nan(a.dbeta, gb, row0 * a.H + hk * r_heads, live, a.H, r_heads, tid, kThreads);
  }
}

template <int NP, int PP>
cudaError_t launch_k(const DeltaArgs &a, cudaStream_t st) {
  using Lay = Layout<NP, PP>;
  auto kern = delta_chunk_grad_kernel<NP, PP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kBytes);
  if (e != cudaSuccess) return e;
  const auto at16 = [](const void *x, const void *y) { return (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % 16 == 0; };
  const dim3 grid((unsigned)((a.L + kChunk - 1) / kChunk), (unsigned)a.Hk, (unsigned)a.Bt);
  kern<<<grid, kThreads, Lay::kBytes, st>>>(a, a.N % 8 == 0 && at16(a.q, a.k), a.P % 8 == 0 && at16(a.dy, a.v), a.N % 8 == 0 && at16(a.dq, a.dk));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chunk_grad(const DeltaArgs &a, cudaStream_t st) {
  cudaError_t e = trace_before(st, "delta_chunk_grad");
  if (e != cudaSuccess) return e;
  if (a.N <= 64) e = a.P <= 64 ? launch_k<64, 64>(a, st) : launch_k<64, 128>(a, st);
  else e = a.P <= 64 ? launch_k<128, 64>(a, st) : launch_k<128, 128>(a, st);
  return e != cudaSuccess ? e : trace_after(st);
}

}  // namespace pdssm
