// The gated delta rule by chunks of 64 steps, first part: what a chunk needs that does
// not depend on the state, for all chunks at once (bf16 inputs; formulas in delta.cuh).
//
// With G_i the running sum of the chunk's log decays, D_ij = exp(G_i - G_j) for j <= i and
// N_ij = D_ij <k_i, k_j> for j < i, the steps of a chunk that starts from H obey
//   (1 + N diag(beta)) e = v - diag(exp G) K H,    du = (1 + diag(beta) N)^-T dU
// (dU: what reaches u = beta e from the outputs and the adjoint behind the chunk). With X
// the solution of (1 + N diag(beta)) X = N, the inverses are
//   Te = (1 + N diag(beta))^-1 = 1 - X diag(beta),  Tb = (1 + diag(beta) N)^-1 = 1 - diag(beta) X,
// one from the other without a division by a beta that may be 0. This kernel writes, per
// value head and chunk, one record: Te, for the backward pass Tb, A_ij = scale D_ij <q_i, k_j>
// (j <= i), and exp(G_i), exp(G_64 - G_i), beta_i, G_i.
// The products of q and k rows are exact in bf16 and summed in fp32: one tensor-core
// product [K; Q] K^T of 128 x 64 a chunk and key head (tcgen05.mma from shared memory,
// M = 128, so that the whole accumulator is used). X is fp32 on the ordinary cores: two
// 32 x 32 triangles, a column a thread in registers, while the other two warps write A;
// then the square below them by two products that skip what is 0. The inverses are
// written as three bf16 parts (24 bits: two would be the largest error of a state that is
// kept in fp32), A as two (the forward pass, where it only reaches an output that is
// rounded to bf16) or three, each in the order of the tensor core's shared-memory operand, so
// that the scan copies a record as it is.
// Measured: 8,192 chunks of 64 x 64: 153 us, 192 with what a backward pass needs (records of 42 and 74
// KiB: 348 and 617 MB, 53 and 94 us of writing); the triangles' chains of FMAs are the rest.
// G is summed in double and kept as two floats: 64 decays can add up to 7,000 while a
// difference next to 0 matters to 2^-24.
#include <algorithm>

#include "delta.cuh"
#include "delta_chunk.cuh"
#include "sm100.cuh"

namespace pdssm {

using namespace sm100;

namespace {

constexpr int kThreads = 128;
constexpr int kLd = kChunk + 4;
constexpr int kGroup = 2 * kChunk * 16 + 16;  // bytes of eight columns of [K; Q]; 16 more spread the banks

// The tile's [K; Q] rows as an operand: rows 0-63 are K, 64-127 are Q.
template <int NP, bool WIDE>
__device__ __forceinline__ void load_rows(uint8_t *dst, const DeltaArgs &a, int64_t row0, int64_t hk, int live) {
  constexpr int G = NP / 8, kStep = kThreads / G;
  const int g = threadIdx.x % G, N = (int)a.N;
  const int64_t row = a.Hk * a.N;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(which ? a.q : a.k) + row0 * row + hk * a.N + 8 * g;
    uint8_t *to = dst + g * kGroup + which * kChunk * 16;
#pragma unroll
    for (int t = threadIdx.x / G; t < kChunk; t += kStep) {
      if (WIDE && t < live && 8 * g < N) cp_async16(to + t * 16, src + t * row);
      else *reinterpret_cast<uint4 *>(to + t * 16) = !WIDE && t < live ? gather8(src + t * row, N - 8 * g) : make_uint4(0, 0, 0, 0);
    }
  }
}

// A step's running log decay in two floats (base 2) and its beta.
struct Gate {
  float hi, lo, beta, pad;
};

__device__ __forceinline__ float decay(float hi, float lo, const Gate &j) { return decay2((hi - j.hi) + (lo - j.lo)); }

// Column j of the 32 x 32 triangle at (o, o): x = N_j - N diag(beta) x by forward substitution,
// nt[j][i] = N_ij. Each known x_m is taken out of the rows below it (independent FMAs).
__device__ __forceinline__ void solve_column(const float *nt, const Gate *gate, int o, int j, float *out) {
  float x[32];
#pragma unroll
  for (int i4 = 0; i4 < 8; ++i4) {
    const float4 v = *reinterpret_cast<const float4 *>(nt + (o + j) * kLd + o + 4 * i4);
    const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int s = 0; s < 4; ++s) x[4 * i4 + s] = 4 * i4 + s > j ? w[s] : 0.f;
  }
#pragma unroll
  for (int m = 1; m < 31; ++m) {
    const float *row = nt + (o + m) * kLd + o;
    const float xm = -gate[o + m].beta * x[m];
#pragma unroll
    for (int i4 = (m + 1) / 4; i4 < 8; ++i4) {
      const float4 v = *reinterpret_cast<const float4 *>(row + 4 * i4);
      const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (4 * i4 + s > m) x[4 * i4 + s] = fmaf(w[s], xm, x[4 * i4 + s]);
    }
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) out[(o + i) * kLd + o + j] = x[i];
}

// 1 - X diag(beta) (Te) or 1 - diag(beta) X (Tb) as three bf16 parts in operand order.
template <bool TB>
__device__ __forceinline__ void write_parts(const float *x, const Gate *gate, uint8_t *dst) {
  const int c = threadIdx.x & (kChunk - 1);
  const float bc = gate[c].beta;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int g = 2 * k + (threadIdx.x >> 6);
    uint32_t p[3][4] = {};
    if (8 * g <= c) {
      const float4 lo = *reinterpret_cast<const float4 *>(x + c * kLd + 8 * g), hi = *reinterpret_cast<const float4 *>(x + c * kLd + 8 * g + 4);
      float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const int j = 8 * g + s;
        v[s] = j < c ? -(TB ? bc : gate[j].beta) * v[s] : j == c ? 1.f : 0.f;
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) split3(v[2 * s], v[2 * s + 1], p[0][s], p[1][s], p[2][s]);
    }
#pragma unroll
    for (int q = 0; q < 3; ++q)
      *reinterpret_cast<uint4 *>(dst + q * kSquare + g * 1024 + c * 16) = make_uint4(p[q][0], p[q][1], p[q][2], p[q][3]);
  }
}

template <int NP>
struct Smem {
  // the operand is read by the tensor core only until its product is done; X then takes its place, and W
  // that of N's upper triangle once it is solved
  static constexpr int kKq = (NP / 8) * kGroup, kX = 4 * kChunk * kLd, kNt = kKq > kX ? kKq : kX;
  static constexpr int kGate = kNt + 4 * kChunk * kLd, kBar = kGate + 16 * kChunk, kBytes = kBar + 16;
};

template <int NP, bool BWD>
__global__ void __launch_bounds__(kThreads, NP == 64 ? 6 : 4) delta_prep_kernel(DeltaArgs a, bool wide) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *kq = smem;
  float *x = reinterpret_cast<float *>(smem), *nt = reinterpret_cast<float *>(smem + Smem<NP>::kNt), *w = nt;
  Gate *gate = reinterpret_cast<Gate *>(smem + Smem<NP>::kGate);
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + Smem<NP>::kBar);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bar + 1);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int64_t chunk = blockIdx.x, hk = blockIdx.y, b = blockIdx.z, t0 = chunk * kChunk;
  const int64_t len = live_steps(a.lengths, b, a.L);
  if (t0 >= len) return;
  const int live = (int)min((int64_t)kChunk, len - t0);
  const int64_t row0 = b * a.L + t0;
  const bool gb = a.gate_t == PDSSM_BF16;
  const int r_heads = (int)(a.H / a.Hk);

  // the gates of a head, two steps a lane of warp 0
  float g[2], be[2];
  const auto fetch_gates = [&](int64_t h) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int c = 2 * lane + s;
      const int64_t at = (row0 + min(c, live - 1)) * a.H + h;
      g[s] = load_any(a.g, at, gb);
      be[s] = load_any(a.beta, at, gb);
    }
  };
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_fence_init();
  }
  if (warp == 0) {
    tmem_alloc(tslot, 64);
    tmem_relinquish();
    fetch_gates(hk * r_heads);
  }
  if (wide) load_rows<NP, true>(kq, a, row0, hk, live);
  else load_rows<NP, false>(kq, a, row0, hk, live);
  cp_async_commit();
  cp_async_wait<0>();
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, *tslot, 0);
  if (warp == 1) {
    constexpr uint32_t id = idesc_bf16_f32(128, kChunk, false, false);
    const uint64_t d = smem_desc(smem_u32(kq), kGroup, 128);
    if (elect_one()) {
#pragma unroll
      for (int ks = 0; ks < NP / 16; ++ks)
        mma_bf16(tbase, d + (ks * 2 * kGroup >> 4), d + (ks * 2 * kGroup >> 4), id, ks > 0);
      mma_commit(bar);
    }
    __syncwarp();
  }

  for (int hh = 0; hh < r_heads; ++hh) {
    const int64_t h = hk * r_heads + hh;
    uint8_t *rec = a.records + ((b * a.H + h) * a.nC + chunk) * a.rec_bytes;
    if (warp == 0) {
      float *scal = reinterpret_cast<float *>(rec + a.rec_bytes - kScalars);
      const double g0 = 2 * lane < live ? (double)clamp_gate(g[0]) * 1.4426950408889634 : 0.0;
      const double g1 = 2 * lane + 1 < live ? (double)clamp_gate(g[1]) * 1.4426950408889634 : 0.0;
      double sum = g0 + g1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      const double last = __shfl_sync(0xffffffffu, sum, 31), G[2] = {sum - g1, sum};
      // the state's decay over the chunk, as a float and what that lacks: hundreds of them are multiplied
      const double all = exp2(last);
      const float2 two = make_float2((float)all, (float)(all - (double)(float)all));
      float grow[2], fade[2], bt[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const float hi = (float)G[s];
        bt[s] = 2 * lane + s < live ? be[s] : 0.f;
        gate[2 * lane + s] = {hi, (float)(G[s] - (double)hi), bt[s], 0.f};
        grow[s] = decay2(hi);
        fade[s] = decay2((float)(last - G[s]));
      }
      float2 *out = reinterpret_cast<float2 *>(scal);
      out[lane] = make_float2(grow[0], grow[1]);
      out[32 + lane] = make_float2(fade[0], fade[1]);
      out[64 + lane] = make_float2(bt[0], bt[1]);
      out[96 + lane] = two;
      out[128 + lane] = make_float2((float)G[0], (float)G[1]);
      out[160 + lane] = make_float2((float)(G[0] - (double)(float)G[0]), (float)(G[1] - (double)(float)G[1]));
      if (hh + 1 < r_heads) fetch_gates(h + 1);
    }
    if (hh == 0) wait_own(bar, 0, a.err);
    __syncthreads();
    tc_fence_after();
    // a thread has one row of the accumulator: rows of K K^T in threads 0-63, of Q K^T in 64-127;
    // rows below 32 end before column 32
    const int i = tid & (kChunk - 1);
    const Gate gi = gate[i];
    if (warp < 2) {
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        if (warp == 0 && part >= 2) break;
        float v[16];
        tmem_ld16(taddr(tbase, 32 * warp, 16 * part), v);
        tmem_wait_ld();
#pragma unroll
        for (int s = 0; s < 16; ++s) {
          const int j = 16 * part + s;
          nt[j * kLd + i] = decay(gi.hi, gi.lo, gate[j]) * v[s];  // read where j < i only
        }
      }
      __syncwarp();
      // a warp's triangle is of its own rows
      solve_column(nt, gate, 32 * warp, lane, x);
    } else {
      uint8_t *dst = rec + (BWD ? 2 : 1) * 3 * kSquare;
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        float v[16];
        const bool none = warp == 2 && part >= 2;
        if (!none) {
          tmem_ld16(taddr(tbase, 32 * warp, 16 * part), v);
          tmem_wait_ld();
        }
#pragma unroll
        for (int s = 0; s < 16; ++s) {
          const int j = 16 * part + s;
          v[s] = !none && j <= i ? a.scale * decay(gi.hi, gi.lo, gate[j]) * v[s] : 0.f;
        }
#pragma unroll
        for (int q8 = 0; q8 < 2; ++q8) {
          uint32_t p[3][4];
#pragma unroll
          for (int s = 0; s < 4; ++s) split3(v[8 * q8 + 2 * s], v[8 * q8 + 2 * s + 1], p[0][s], p[1][s], p[2][s]);
#pragma unroll
          for (int q = 0; q < delta_a_parts(BWD); ++q)
            *reinterpret_cast<uint4 *>(dst + q * kSquare + (2 * part + q8) * 1024 + i * 16) =
                make_uint4(p[q][0], p[q][1], p[q][2], p[q][3]);
        }
      }
    }
    __syncthreads();
    // The square below the triangles: W = N21 (1 - diag(beta1) X11), X21 = W - X22 diag(beta2) W.
    {
      // columns 8 warp .. + 7 of row `lane`; X11 starts below its diagonal
      float acc[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) acc[s] = nt[(8 * warp + s) * kLd + 32 + lane];
#pragma unroll 4
      for (int m = 8 * warp + 1; m < 32; ++m) {
        const float l = -nt[m * kLd + 32 + lane] * gate[m].beta;
        const float4 u = *reinterpret_cast<const float4 *>(x + m * kLd + 8 * warp), v = *reinterpret_cast<const float4 *>(x + m * kLd + 8 * warp + 4);
        acc[0] = fmaf(l, u.x, acc[0]); acc[1] = fmaf(l, u.y, acc[1]); acc[2] = fmaf(l, u.z, acc[2]); acc[3] = fmaf(l, u.w, acc[3]);
        acc[4] = fmaf(l, v.x, acc[4]); acc[5] = fmaf(l, v.y, acc[5]); acc[6] = fmaf(l, v.z, acc[6]); acc[7] = fmaf(l, v.w, acc[7]);
      }
      *reinterpret_cast<float4 *>(w + lane * kLd + 8 * warp) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      *reinterpret_cast<float4 *>(w + lane * kLd + 8 * warp + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
    __syncthreads();
    {
      // rows 8 warp .. + 7 of column `lane`; X22 ends before its diagonal
      float acc[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) acc[r] = w[(8 * warp + r) * kLd + lane];
#pragma unroll 2
      for (int m = 0; m < 8 * warp + 8; m += 4) {
        float u[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) u[s] = -gate[32 + m + s].beta * w[(m + s) * kLd + lane];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float4 v = *reinterpret_cast<const float4 *>(x + (32 + 8 * warp + r) * kLd + 32 + m);
          acc[r] = fmaf(v.x, u[0], fmaf(v.y, u[1], fmaf(v.z, u[2], fmaf(v.w, u[3], acc[r]))));
        }
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) x[(32 + 8 * warp + r) * kLd + lane] = acc[r];
    }
    __syncthreads();
    write_parts<false>(x, gate, rec);
    if (BWD) write_parts<true>(x, gate, rec + 3 * kSquare);
    __syncthreads();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tbase, 64);
}

template <int NP, bool BWD>
cudaError_t launch_n(const DeltaArgs &a, cudaStream_t st) {
  const size_t smem = Smem<NP>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(delta_prep_kernel<NP, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const bool wide = a.N % 8 == 0 && reinterpret_cast<uintptr_t>(a.q) % 16 == 0 && reinterpret_cast<uintptr_t>(a.k) % 16 == 0;
  const dim3 grid((unsigned)a.nC, (unsigned)a.Hk, (unsigned)a.Bt);
  delta_prep_kernel<NP, BWD><<<grid, kThreads, smem, st>>>(a, wide);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_prep(const DeltaArgs &a, bool bwd, cudaStream_t st) {
  cudaError_t e = trace_before(st, "delta_prep");
  if (e != cudaSuccess) return e;
  if (a.N <= 64) e = bwd ? launch_n<64, true>(a, st) : launch_n<64, false>(a, st);
  else e = bwd ? launch_n<128, true>(a, st) : launch_n<128, false>(a, st);
  return e != cudaSuccess ? e : trace_after(st);
}

}  // namespace pdssm
