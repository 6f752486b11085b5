// Gradients of queries, keys, decays and betas of the gated delta rule, chunk by chunk
// in parallel, once the states before the chunks (H), the adjoints behind them (X), e
// and du are known (csrc/delta_steps.cu, csrc/delta_rows.cu).
//
// For the chunk's rows i, j with G the running sum of its log decays, D_ij = exp(G_i - G_j)
// for j <= i, gam_i = exp(G_i), last = exp(G_C), fade_i = exp(G_C - G_i), u = beta e, qs = scale q:
//   F1_ij = D_ij <dy_i, u_j>             (j <= i)
//   F2_ij = -beta_i D_ij <du_i, u_j>     (j < i)
//   dq_i  = scale (gam_i H dy_i + sum_j F1_ij k_j)
//   dk_i  = fade_i X u_i - beta_i gam_i H du_i + sum_j F1_ji qs_j + sum_j (F2_ij + F2_ji) k_j
//   dbeta_i = <du_i, e_i>
//   dG_i  = <qs_i, gam_i H dy_i> - <k_i, beta_i gam_i H du_i>
//           + sum_j (F1_ij <qs_i, k_j> + F2_ij <k_i, k_j>) - sum_j (F1_ji <qs_j, k_i> + F2_ji <k_j, k_i>)   (j < i, j > i)
//   dg_i  = sum of dG_j over j >= i + last <X, H> + sum over j < i of <k_j, fade_j X u_j>
// Every term has a factor exp(g); those of pairs behind step i cancel in dg_i up to their rounding (so where exp(g_i)
// is 0 in fp32, dg_i is set to 0).
//
// A block has one chunk of 32 steps of one key head and goes through the value heads
// that share it, so their sum for dq and dk stays in registers and needs neither
// atomics nor a second pass. All products are fp32 from shared memory: a thread holds
// 4 rows and every 32nd column, rows are padded to an odd number of 16-byte pieces, so
// the loads of a warp are broadcasts or free of conflicts. It is bound by those loads
// (about 20 for 64 FMAs of a warp).
#include <algorithm>

#include "delta.cuh"

namespace pdssm {

namespace {

constexpr int kC = 32, kThreads = 256, kLdF = kC + 4;

__host__ __device__ constexpr int odd_pieces(int n) { return 4 * (((n + 3) / 4) | 1); }

struct Shape {
  int ldn, ldp, rows;  // row lengths of the q / k and of the p-wide arrays; rows of the state's buffer
  size_t bytes;
};

Shape shape_of(int J, int64_t N, int64_t Pp) {
  Shape s;
  s.ldn = odd_pieces(32 * J);
  s.ldp = odd_pieces((int)Pp);
  s.rows = 32 * J;
  s.bytes = 4 * ((size_t)2 * kC * s.ldn + 3 * kC * s.ldp + (size_t)s.rows * s.ldp + 2 * kC * kLdF + 8 * kC + 8 * kC + 16);
  return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

// acc[r][j] += sum_p rows[4 ty + r][p] m[tx + 32 j][p]
template <int J>
__device__ __forceinline__ void rows_by_state(float (&acc)[4][J], const float *rows, const float *m, int ld, int Pp, int ty, int tx) {
  for (int p = 0; p < Pp; p += 4) {
    float4 x[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = *reinterpret_cast<const float4 *>(rows + (4 * ty + r) * ld + p);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float4 v = *reinterpret_cast<const float4 *>(m + (tx + 32 * j) * ld + p);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r][j] = dot4(x[r], v, acc[r][j]);
    }
  }
}

// acc[r][j] += sum_i f[4 ty + r][i] (or f[i][4 ty + r] with T) m[i][tx + 32 j]
template <int J, bool TR>
__device__ __forceinline__ void square_by_rows(float (&acc)[4][J], const float *f, const float *m, int ld, int ty, int tx) {
#pragma unroll 2
  for (int i = 0; i < kC; i += 4) {
    float w[4][4];  // [row r][i + s]
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float4 v = *reinterpret_cast<const float4 *>(TR ? f + (i + s) * kLdF + 4 * ty : f + (4 * ty + s) * kLdF + i);
      if (TR) { w[0][s] = v.x; w[1][s] = v.y; w[2][s] = v.z; w[3][s] = v.w; }
      else { w[s][0] = v.x; w[s][1] = v.y; w[s][2] = v.z; w[s][3] = v.w; }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float x = m[(i + s) * ld + tx + 32 * j];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r][j] = fmaf(w[r][s], x, acc[r][j]);
      }
  }
}

template <int J>
__global__ void __launch_bounds__(kThreads) delta_grad_kernel(DeltaArgs a, int ldn, int ldp) {
  extern __shared__ __align__(16) float smem[];
  const bool bf = a.in_t == PDSSM_BF16, gb = a.gate_t == PDSSM_BF16;
  const int N = (int)a.N, P = (int)a.P, Pp = (int)a.Pp;
  float *Q = smem, *K = Q + kC * ldn, *Y = K + kC * ldn, *U = Y + kC * ldp, *R = U + kC * ldp, *M = R + kC * ldp;
  float *F1 = M + 32 * J * ldp, *F2 = F1 + kC * kLdF, *colp = F2 + kC * kLdF;
  float *sb = colp + 8 * kC, *sgam = sb + kC, *sfade = sgam + kC, *sdG = sfade + kC, *sdb = sdG + kC, *shi = sdb + kC,
        *slo = shi + kC, *sx = slo + kC, *swarp = sx + kC;
  const int tid = threadIdx.x, ty = tid >> 5, tx = tid & 31;
  const int64_t chunk = blockIdx.x, hk = blockIdx.y, b = blockIdx.z, t0 = chunk * kC;
  const int r_heads = (int)(a.H / a.Hk);
  const int64_t len = live_steps(a.lengths, b, a.L);
  const int rows = (int)min((int64_t)kC, a.L - t0), live = (int)max((int64_t)0, min((int64_t)kC, len - t0));
  const int64_t row0 = b * a.L + t0;
  if (live == 0) {
    for (int i = tid; i < rows * N; i += kThreads) {
      const int64_t at = ((row0 + i / N) * a.Hk + hk) * N + i % N;
      store_any(a.dq, at, bf, 0.f);
      store_any(a.dk, at, bf, 0.f);
    }
    for (int i = tid; i < rows * r_heads; i += kThreads) {
      const int64_t at = (row0 + i / r_heads) * a.H + hk * r_heads + i % r_heads;
      store_any(a.dg, at, gb, 0.f);
      store_any(a.dbeta, at, gb, 0.f);
    }
    return;
  }
  if (tid == 0) swarp[9] = timed_out(a.err) ? 1.f : 0.f;
  for (int i = tid; i < kC * 32 * J; i += kThreads) {
    const int t = i / (32 * J), n = i % (32 * J);
    const bool on = t < live && n < N;
    const int64_t at = ((row0 + t) * a.Hk + hk) * N + n;
    Q[t * ldn + n] = on ? load_any(a.q, at, bf) * a.scale : 0.f;
    K[t * ldn + n] = on ? load_any(a.k, at, bf) : 0.f;
  }
  __syncthreads();
  float qk[4] = {}, kk[4] = {};  // <qs_i, k_j>, <k_i, k_j> for i = 4 ty + r, j = tx
  for (int n = 0; n < 32 * J; n += 4) {
    const float4 kj = *reinterpret_cast<const float4 *>(K + tx * ldn + n);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      qk[r] = dot4(*reinterpret_cast<const float4 *>(Q + (4 * ty + r) * ldn + n), kj, qk[r]);
      kk[r] = dot4(*reinterpret_cast<const float4 *>(K + (4 * ty + r) * ldn + n), kj, kk[r]);
    }
  }
  float dq[4][J] = {}, dk[4][J] = {};
  for (int hh = 0; hh < r_heads; ++hh) {
    const int64_t h = hk * r_heads + hh, bh = b * a.H + h;
    const float *carry = a.carry + (bh * a.nC + chunk) * N * Pp, *xcarry = a.xcarry + (bh * a.nC + chunk) * N * Pp;
    __syncthreads();  // the arrays of the head before have been read
    bool dropped = false;  // warp 0: the state before its step does not matter
    if (ty == 0) {
      const int64_t at = (row0 + tx) * a.H + h;
      const float g = tx < live ? clamp_gate(load_any(a.g, at, gb)) : 0.f;
      dropped = expf(g) == 0.f;
      double G = (double)g;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, G, o);
        if (tx >= o) G += up;
      }
      const double Gl = __shfl_sync(0xffffffffu, G, 31);
      sb[tx] = tx < live ? load_any(a.beta, at, gb) : 0.f;
      sgam[tx] = expf((float)G);
      sfade[tx] = expf((float)(Gl - G));
      shi[tx] = (float)G;
      slo[tx] = (float)(G - (double)(float)G);
      if (tx == 31) swarp[8] = expf((float)Gl);
    }
    for (int i = tid; i < kC * Pp; i += kThreads) {
      const int t = i / Pp, p = i % Pp;
      const int64_t at = (row0 + t) * a.H + h;
      Y[t * ldp + p] = (t < live && p < P) ? load_any(a.dy, at * P + p, bf) : 0.f;
      const int64_t row = bh * a.L + t0 + t;
      U[t * ldp + p] = t < live ? a.e[row * Pp + p] : 0.f;
      R[t * ldp + p] = t < live ? a.du[row * Pp + p] : 0.f;
    }
    for (int i = tid; i < 32 * J * Pp; i += kThreads) {
      const int n = i / Pp, p = i % Pp;
      M[n * ldp + p] = n < N ? carry[n * Pp + p] : 0.f;
    }
    __syncthreads();
    // dbeta, and u in the place of e: a warp has rows 4 ty .. + 3
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 4 * ty + r;
      float s = 0.f;
      for (int p = tx; p < Pp; p += 32) {
        s = fmaf(U[t * ldp + p], R[t * ldp + p], s);
        U[t * ldp + p] *= sb[t];
      }
      s = warp_sum(s);
      if (tx == 0) sdb[t] = s;
    }
    __syncthreads();
    // the squares, and their part of dG
    {
      float yu[4] = {}, ru[4] = {};
      for (int p = 0; p < Pp; p += 4) {
        const float4 u = *reinterpret_cast<const float4 *>(U + tx * ldp + p);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          yu[r] = dot4(*reinterpret_cast<const float4 *>(Y + (4 * ty + r) * ldp + p), u, yu[r]);
          ru[r] = dot4(*reinterpret_cast<const float4 *>(R + (4 * ty + r) * ldp + p), u, ru[r]);
        }
      }
      float col = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 4 * ty + r, j = tx;
        float f1 = 0.f, f2 = 0.f;
        if (j <= i) {
          const float D = expf((shi[i] - shi[j]) + (slo[i] - slo[j]));
          f1 = D * yu[r];
          if (j < i) f2 = -sb[i] * D * ru[r];
        }
        F1[i * kLdF + j] = f1;
        if (j < i) F2[i * kLdF + j] = F2[j * kLdF + i] = f2;
        if (j == i) F2[i * kLdF + j] = 0.f;
        const float w = j < i ? f1 * qk[r] + f2 * kk[r] : 0.f;
        col += w;
        const float s = warp_sum(w);
        if (tx == 0) sdG[i] = s;
      }
      colp[ty * kC + tx] = col;
    }
    __syncthreads();
    square_by_rows<J, false>(dq, F1, K, ldn, ty, tx);
    square_by_rows<J, true>(dk, F1, Q, ldn, ty, tx);
    square_by_rows<J, false>(dk, F2, K, ldn, ty, tx);
    float alpha[4] = {};
    {
      float t[4][J] = {};
      rows_by_state<J>(t, Y, M, ldp, Pp, ty, tx);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float gam = sgam[4 * ty + r];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float v = gam * t[r][j];
          dq[r][j] += v;
          alpha[r] = fmaf(Q[(4 * ty + r) * ldn + tx + 32 * j], v, alpha[r]);
        }
      }
    }
    {
      float t[4][J] = {};
      rows_by_state<J>(t, R, M, ldp, Pp, ty, tx);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float f = -sb[4 * ty + r] * sgam[4 * ty + r];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float v = f * t[r][j];
          dk[r][j] += v;
          alpha[r] = fmaf(K[(4 * ty + r) * ldn + tx + 32 * j], v, alpha[r]);
        }
      }
    }
    __syncthreads();
    // X in the place of H, and <X, H>
    float xh = 0.f;
    for (int i = tid; i < 32 * J * Pp; i += kThreads) {
      const int n = i / Pp, p = i % Pp;
      const float x = n < N ? xcarry[n * Pp + p] : 0.f;
      xh = fmaf(x, M[n * ldp + p], xh);
      M[n * ldp + p] = x;
    }
    xh = warp_sum(xh);
    if (tx == 0) swarp[ty] = xh;
    __syncthreads();
    {
      float t[4][J] = {};
      rows_by_state<J>(t, U, M, ldp, Pp, ty, tx);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 4 * ty + r;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float v = sfade[i] * t[r][j];
          dk[r][j] += v;
          s = fmaf(K[i * ldn + tx + 32 * j], v, s);
        }
        s = warp_sum(s);
        const float al = warp_sum(alpha[r]);
        if (tx == 0) {
          sx[i] = s;
          sdG[i] += al;
        }
      }
    }
    __syncthreads();
    if (ty == 0) {
      // the suffix sums of dG, the sums of what goes out of the earlier steps (those of all steps less the suffix
      // would leave the rounding of the last one's, which has no factor), and the state's way through the chunk
      float d = sdG[tx], xhs = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        d -= colp[w * kC + tx];
        xhs += swarp[w];
      }
      double s = (double)d, out = __shfl_up_sync(0xffffffffu, sx[tx], 1);
      if (tx == 0) out = 0.0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double dn = __shfl_down_sync(0xffffffffu, s, o), up = __shfl_up_sync(0xffffffffu, out, o);
        if (tx + o < 32) s += dn;
        if (tx >= o) out += up;
      }
      s += out + (double)(swarp[8] * xhs);
      if (tx < rows) {
        const int64_t at = (row0 + tx) * a.H + h;
        store_any(a.dg, at, gb, tx < live && !dropped ? (float)s : 0.f);
        store_any(a.dbeta, at, gb, tx < live ? sdb[tx] : 0.f);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int t = 4 * ty + r;
    if (t >= rows) continue;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int n = tx + 32 * j;
      if (n >= N) continue;
      const int64_t at = ((row0 + t) * a.Hk + hk) * N + n;
      store_any(a.dq, at, bf, t < live ? a.scale * dq[r][j] : 0.f);
      store_any(a.dk, at, bf, t < live ? dk[r][j] : 0.f);
    }
  }
  __syncthreads();
  if (swarp[9] != 0.f) {
    fill_nan(a.dq, bf, (row0 * a.Hk + hk) * N, live, a.Hk * N, N, tid, kThreads);
    fill_nan(a.dk, bf, (row0 * a.Hk + hk) * N, live, a.Hk * N, N, tid, kThreads);
    fill_nan(a.dg, gb, row0 * a.H + hk * r_heads, live, a.H, r_heads, tid, kThreads);
    fill_nan(a.dbeta, gb, row0 * a.H + hk * r_heads, live, a.H, r_heads, tid, kThreads);
  }
}

template <int J>
cudaError_t launch_j(const DeltaArgs &a, cudaStream_t st) {
  const Shape s = shape_of(J, a.N, a.Pp);
  cudaError_t e = allow_shared(delta_grad_kernel<J>);
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((a.L + kC - 1) / kC), (unsigned)a.Hk, (unsigned)a.Bt);
  delta_grad_kernel<J><<<grid, kThreads, s.bytes, st>>>(a, s.ldn, s.ldp);
  return cudaGetLastError();
}

}  // namespace

int64_t delta_grad_chunk() { return kC; }

cudaError_t launch_delta_grad(const DeltaArgs &a, cudaStream_t st) {
  cudaError_t e = trace_before(st, "delta_grad");
  if (e != cudaSuccess) return e;
  e = a.N <= 32 ? launch_j<1>(a, st) : a.N <= 64 ? launch_j<2>(a, st) : launch_j<4>(a, st);
  return e != cudaSuccess ? e : trace_after(st);
}

}  // namespace pdssm
