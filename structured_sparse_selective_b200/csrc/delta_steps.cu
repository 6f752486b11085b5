// The gated delta rule step by step (formulas in delta.cuh), forwards and backwards:
// single tokens and short runs, fp32 inputs, and every size.
//
// The columns of H are independent of one another. A warp owns 16 columns: lane
// (rg, cl) = (lane / 4, lane % 4) holds columns 4 cl .. 4 cl + 3 and rows
// 32 j + 4 rg .. + 3 in registers for the whole sequence, so the state moves once in
// and once out. k^T H is a sum over the lane's rows and three shuffles over the eight
// row groups; no barrier joins the warps but the one a tile of 8 steps has, whose
// k, q, v, decay and beta a loader warp brings to shared memory in fp32 while the
// others work on the tile before.
// A step's products are in row pairs (fma.rn.f32x2), which halves the instructions.
// What bounds it: for one step the state's bytes (read and written once); for long
// sequences the chain dot -> shuffles -> update of each step, and with enough
// sequences the issue rate of its ~140 instructions a warp.
#include <algorithm>

#include "delta.cuh"

namespace pdssm {

namespace {

constexpr int kTS = 8;        // steps a tile
constexpr int kWarpCols = 16;
constexpr int kMaxWarps = PDSSM_MAX_P / kWarpCols;

// One tile in shared memory: rows of k and q (padded with zeros to 32 J), of the
// block's columns of v (or dy), and (a, beta).
template <int J>
struct Tile {
  static constexpr int kRow = 32 * J;
  float *k, *q, *c;
  float2 *ab;
  __device__ Tile(float *base, int cols, int buf) {
    const int one = kTS * (2 * kRow + cols + 2);
    base += buf * one;
    k = base;
    q = base + kTS * kRow;
    c = base + 2 * kTS * kRow;
    ab = reinterpret_cast<float2 *>(c + kTS * cols);
  }
  static size_t bytes(int cols) { return (size_t)2 * kTS * (2 * kRow + cols + 2) * 4; }
};

// The loader warp. A tile's values wait in registers while the tile before is computed:
// fetch() starts the loads of one tile, put() writes them to shared memory a tile later,
// so HBM's latency is behind a whole tile's work. The loads are unconditional, from a
// valid place where there is nothing to load: with a branch around each they ran one
// after the other (LM layer: 1.9 ms).
template <int J, typename T, typename G>
struct Loader {
  static constexpr int M = kMaxWarps / 2;
  const DeltaArgs &a;
  const T *k, *q, *c;
  const G *g, *beta;
  int lane, p0, cols, n;
  int64_t rowk, rowc;
  T kv[kTS][J], qv[kTS][J], cv[kTS][M];
  G gv, bv;

  // `src`: v forwards, dy backwards.
  __device__ Loader(const DeltaArgs &a_, int64_t b, int64_t h, int p0_, int cols_, const void *src)
      : a(a_), lane(threadIdx.x & 31), p0(p0_), cols(cols_), n(0), rowk(a_.Hk * a_.N), rowc(a_.H * a_.P) {
    const int64_t hk = h / (a.H / a.Hk);
    k = static_cast<const T *>(a.k) + b * a.L * rowk + hk * a.N;
    q = static_cast<const T *>(a.q) + b * a.L * rowk + hk * a.N;
    c = static_cast<const T *>(src) + b * a.L * rowc + h * a.P;
    g = static_cast<const G *>(a.g) + b * a.L * a.H + h;
    beta = static_cast<const G *>(a.beta) + b * a.L * a.H + h;
  }

  // Steps [t0, t0 + steps), steps <= kTS; nothing for steps <= 0.
  __device__ __forceinline__ void fetch(int64_t t0, int64_t steps) {
    n = (int)(steps < kTS ? steps : kTS);
    if (n <= 0) return;
#pragma unroll
    for (int s = 0; s < kTS; ++s) {
      const int64_t t = t0 + min(s, n - 1);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int i = min(lane + 32 * j, (int)a.N - 1);
        kv[s][j] = k[t * rowk + i];
        qv[s][j] = q[t * rowk + i];
      }
#pragma unroll
      for (int j = 0; j < M; ++j) cv[s][j] = c[t * rowc + min(p0 + min(lane + 32 * j, cols - 1), (int)a.P - 1)];
    }
    const int64_t t = (t0 + min(lane, n - 1)) * a.H;
    gv = g[t];
    bv = beta[t];
  }

  __device__ __forceinline__ void put(const Tile<J> &tile) {
    if (n <= 0) return;
#pragma unroll
    for (int s = 0; s < kTS; ++s) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int i = lane + 32 * j;
        tile.k[s * 32 * J + i] = i < a.N ? to_f32(kv[s][j]) : 0.f;
        tile.q[s * 32 * J + i] = i < a.N ? to_f32(qv[s][j]) * a.scale : 0.f;
      }
#pragma unroll
      for (int j = 0; j < M; ++j) {
        const int i = lane + 32 * j;
        if (i < cols) tile.c[s * cols + i] = p0 + i < a.P ? to_f32(cv[s][j]) : 0.f;
      }
    }
    if (lane < kTS) tile.ab[lane] = make_float2(expf(clamp_gate(to_f32(gv))), to_f32(bv));
  }
};

// The lane's part of a state [N][P] at `p` (null: zeros), in row pairs.
template <int J>
__device__ __forceinline__ void load_state(pair2 (&h)[2 * J][4], const float *p, int64_t N, int64_t P, int64_t ld, int rg, int col) {
  const bool wide = ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    float v[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t n = 32 * j + 4 * rg + r;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[r][c] = 0.f;
      if (p && n < N) {
        if (wide && col + 3 < P) {
          const float4 x = *reinterpret_cast<const float4 *>(p + n * ld + col);
          v[r][0] = x.x; v[r][1] = x.y; v[r][2] = x.z; v[r][3] = x.w;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (col + c < P) v[r][c] = p[n * ld + col + c];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      h[2 * j][c] = pack2(v[0][c], v[1][c]);
      h[2 * j + 1][c] = pack2(v[2][c], v[3][c]);
    }
  }
}

template <int J>
__device__ __forceinline__ void store_state(const pair2 (&h)[2 * J][4], float *p, int64_t N, int64_t P, int64_t ld, int rg, int col) {
  const bool wide = ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    float v[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      unpack2(h[2 * j][c], v[0][c], v[1][c]);
      unpack2(h[2 * j + 1][c], v[2][c], v[3][c]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t n = 32 * j + 4 * rg + r;
      if (n >= N) continue;
      if (wide && col + 3 < P) {
        *reinterpret_cast<float4 *>(p + n * ld + col) = make_float4(v[r][0], v[r][1], v[r][2], v[r][3]);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (col + c < P) p[n * ld + col + c] = v[r][c];
      }
    }
  }
}

// The lane's four rows a j of a vector in shared memory, as pairs.
template <int J>
__device__ __forceinline__ void load_rows(pair2 (&x)[2 * J], const float *p, int rg) {
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float4 v = *reinterpret_cast<const float4 *>(p + 32 * j + 4 * rg);
    x[2 * j] = pack2(v.x, v.y);
    x[2 * j + 1] = pack2(v.z, v.w);
  }
}

// s[c] = sum over the lane's rows of x h[c].
template <int J>
__device__ __forceinline__ void dot_rows(float (&s)[4], const pair2 (&x)[2 * J], const pair2 (&h)[2 * J][4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    pair2 p = mul2(x[0], h[0][c]);
#pragma unroll
    for (int i = 1; i < 2 * J; ++i) p = fma2(x[i], h[i][c], p);
    float u, w;
    unpack2(p, u, w);
    s[c] = u + w;
  }
}

// Sum over the eight row groups, in every lane.
__device__ __forceinline__ void sum_groups(float (&s)[4]) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[c] += __shfl_xor_sync(0xffffffffu, s[c], o);
}

// Sum over the eight row groups of column c = 2 (lane >> 4) + (lane >> 3 & 1) of the
// lane's four: four shuffles instead of twelve where one lane needs one column.
__device__ __forceinline__ float sum_groups_one(const float (&s)[4], int lane) {
  const bool up = lane & 16, mid = lane & 8;
  const float a = (up ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, up ? s[0] : s[2], 16);
  const float b = (up ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, up ? s[1] : s[3], 16);
  float r = (mid ? b : a) + __shfl_xor_sync(0xffffffffu, mid ? a : b, 8);
  return r + __shfl_xor_sync(0xffffffffu, r, 4);
}

// grid: (column groups, heads, batch); warps 0 .. warps - 1 compute, the last loads.
// SAVE: writes e_t and, every a.C steps, the state before them (for the backward pass).
template <int J, typename T, typename G, bool SAVE>
__global__ void __launch_bounds__(32 * (kMaxWarps + 1)) delta_steps_kernel(DeltaArgs a) {
  extern __shared__ __align__(16) float smem[];
  const int warps = blockDim.x / 32 - 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = lane >> 2, cols = warps * kWarpCols, p0 = blockIdx.x * cols;
  const int64_t h = blockIdx.y, b = blockIdx.z, bh = b * a.H + h;
  const int64_t len = live_steps(a.lengths, b, a.L);
  const int col = p0 + warp * kWarpCols + 4 * (lane & 3);
  const bool loader = warp == warps;
  if (loader) {
    Loader<J, T, G> in(a, b, h, p0, cols, a.v);
    in.fetch(0, len);
    in.put(Tile<J>(smem, cols, 0));
    in.fetch(kTS, len - kTS);
    __syncthreads();
    for (int64_t t0 = 0, i = 0; t0 < len; t0 += kTS, ++i) {
      in.put(Tile<J>(smem, cols, (i + 1) & 1));
      in.fetch(t0 + 2 * kTS, len - t0 - 2 * kTS);
      __syncthreads();
    }
    return;
  }
  pair2 st[2 * J][4];
  load_state<J>(st, a.h0 ? a.h0 + bh * a.N * a.P : nullptr, a.N, a.P, a.P, rg, col);
  __syncthreads();
  const int yc = 2 * (lane >> 4) + ((lane >> 3) & 1);
  T *y = static_cast<T *>(a.y);
  for (int64_t t0 = 0, i = 0; t0 < len; t0 += kTS, ++i) {
    const Tile<J> tile(smem, cols, i & 1);
    const int n = (int)min((int64_t)kTS, len - t0);
    for (int s = 0; s < n; ++s) {
      if (SAVE && ((t0 + s) & (a.C - 1)) == 0)
        store_state<J>(st, a.carry + (bh * a.nC + (t0 + s) / a.C) * a.N * a.Pp, a.N, a.Pp, a.Pp, rg, col);
      pair2 k[2 * J], q[2 * J];
      load_rows<J>(k, tile.k + s * 32 * J, rg);
      load_rows<J>(q, tile.q + s * 32 * J, rg);
      const float4 v4 = *reinterpret_cast<const float4 *>(tile.c + s * cols + warp * kWarpCols + 4 * (lane & 3));
      const float2 ab = tile.ab[s];
      float d[4], e[4];
      dot_rows<J>(d, k, st);
      sum_groups(d);
      e[0] = fmaf(-ab.x, d[0], v4.x); e[1] = fmaf(-ab.x, d[1], v4.y);
      e[2] = fmaf(-ab.x, d[2], v4.z); e[3] = fmaf(-ab.x, d[3], v4.w);
      const int64_t row = (b * a.L + t0 + s) * a.H + h;
      if (SAVE && lane < 4 && col < a.Pp)
        *reinterpret_cast<float4 *>(a.e + row * a.Pp + col) = make_float4(e[0], e[1], e[2], e[3]);
      const pair2 aa = pack2(ab.x, ab.x);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float u = ab.y * e[c];
        const pair2 uu = pack2(u, u);
#pragma unroll
        for (int r = 0; r < 2 * J; ++r) st[r][c] = fma2(k[r], uu, mul2(aa, st[r][c]));
      }
      if (!SAVE) {
        float z[4];
        dot_rows<J>(z, q, st);
        const float out = sum_groups_one(z, lane);
        if (!(lane & 4) && col + yc < a.P) st_out(y + row * a.P + col + yc, out);
      }
    }
    __syncthreads();
  }
  if (!SAVE) {
    for (int64_t t = len + rg; t < a.L; t += 8)
      for (int c = 0; c < 4; ++c)
        if (col + c < a.P) st_out(y + ((b * a.L + t) * a.H + h) * a.P + col + c, 0.f);
    if (a.h_final) store_state<J>(st, a.h_final + bh * a.N * a.P, a.N, a.P, a.P, rg, col);
  }
}

// The adjoint X runs from the last step to the first; writes dv_t, du_t, X' at the end
// of each chunk of a.C steps, and dh0.
template <int J, typename T, typename G>
__global__ void __launch_bounds__(32 * (kMaxWarps + 1)) delta_steps_bwd_kernel(DeltaArgs a) {
  extern __shared__ __align__(16) float smem[];
  const int warps = blockDim.x / 32 - 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rg = lane >> 2, cols = warps * kWarpCols, p0 = blockIdx.x * cols;
  const int64_t h = blockIdx.y, b = blockIdx.z, bh = b * a.H + h;
  const int64_t len = live_steps(a.lengths, b, a.L);
  const int col = p0 + warp * kWarpCols + 4 * (lane & 3);
  const bool loader = warp == warps;
  const int64_t tiles = (len + kTS - 1) / kTS;
  if (loader) {
    Loader<J, T, G> in(a, b, h, p0, cols, a.dy);
    const auto fetch = [&](int64_t i) {  // the i-th tile from the end; nothing behind the first
      const int64_t t0 = (tiles - 1 - i) * kTS;
      in.fetch(t0, i < tiles ? len - t0 : 0);
    };
    fetch(0);
    in.put(Tile<J>(smem, cols, 0));
    fetch(1);
    __syncthreads();
    for (int64_t i = 0; i < tiles; ++i) {
      in.put(Tile<J>(smem, cols, (i + 1) & 1));
      fetch(i + 2);
      __syncthreads();
    }
    return;
  }
  pair2 st[2 * J][4];
  load_state<J>(st, a.dh_final ? a.dh_final + bh * a.N * a.P : nullptr, a.N, a.P, a.P, rg, col);
  __syncthreads();
  T *dv = static_cast<T *>(a.dv);
  for (int64_t i = 0; i < tiles; ++i) {
    const int64_t t0 = (tiles - 1 - i) * kTS;
    const Tile<J> tile(smem, cols, i & 1);
    const int n = (int)min((int64_t)kTS, len - t0);
    for (int s = n - 1; s >= 0; --s) {
      const int64_t t = t0 + s;
      if (t == len - 1 || ((t + 1) & (a.C - 1)) == 0)
        store_state<J>(st, a.xcarry + (bh * a.nC + t / a.C) * a.N * a.Pp, a.N, a.Pp, a.Pp, rg, col);
      pair2 k[2 * J], q[2 * J];
      load_rows<J>(k, tile.k + s * 32 * J, rg);
      load_rows<J>(q, tile.q + s * 32 * J, rg);
      const float4 d4 = *reinterpret_cast<const float4 *>(tile.c + s * cols + warp * kWarpCols + 4 * (lane & 3));
      const float2 ab = tile.ab[s];
      const float dy[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const pair2 dd = pack2(dy[c], dy[c]);
#pragma unroll
        for (int r = 0; r < 2 * J; ++r) st[r][c] = fma2(q[r], dd, st[r][c]);
      }
      float du[4];
      dot_rows<J>(du, k, st);
      sum_groups(du);
      const int64_t row = (b * a.L + t) * a.H + h;
      const pair2 aa = pack2(ab.x, ab.x);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float w = -ab.y * du[c];
        const pair2 ww = pack2(w, w);
#pragma unroll
        for (int r = 0; r < 2 * J; ++r) st[r][c] = mul2(aa, fma2(k[r], ww, st[r][c]));
      }
      if (lane < 4 && col < a.Pp) {
        *reinterpret_cast<float4 *>(a.du + row * a.Pp + col) = make_float4(du[0], du[1], du[2], du[3]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (col + c < a.P) st_out(dv + row * a.P + col + c, ab.y * du[c]);
      }
    }
    __syncthreads();
  }
  for (int64_t t = len + rg; t < a.L; t += 8)
    for (int c = 0; c < 4; ++c)
      if (col + c < a.P) st_out(dv + ((b * a.L + t) * a.H + h) * a.P + col + c, 0.f);
  if (a.dh0) store_state<J>(st, a.dh0 + bh * a.N * a.P, a.N, a.P, a.P, rg, col);
}

enum Which { kForward, kForwardSave, kBackward };

template <int J, typename T, typename G>
cudaError_t launch_jtg(const DeltaArgs &a, Which which, cudaStream_t st) {
  // all columns of a head in one block share its loaded tiles; with few sequences the
  // columns are spread over more blocks, down to one warp, until there is one an SM
  int warps = (int)((a.P + kWarpCols - 1) / kWarpCols);
  const int64_t all = warps;
  while (warps > 1 && a.Bt * a.H * ((all + warps - 1) / warps) < 148) warps = (warps + 1) / 2;
  const dim3 grid((unsigned)((all + warps - 1) / warps), (unsigned)a.H, (unsigned)a.Bt);
  const size_t smem = Tile<J>::bytes(warps * kWarpCols);
  auto kern = which == kForward ? delta_steps_kernel<J, T, G, false>
                                : which == kForwardSave ? delta_steps_kernel<J, T, G, true> : delta_steps_bwd_kernel<J, T, G>;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<grid, 32 * (warps + 1), smem, st>>>(a);
  return cudaGetLastError();
}

template <int J>
cudaError_t launch_j(const DeltaArgs &a, Which which, cudaStream_t st) {
  const bool bf = a.in_t == PDSSM_BF16, gb = a.gate_t == PDSSM_BF16;
  using H = __nv_bfloat16;
  if (bf) return gb ? launch_jtg<J, H, H>(a, which, st) : launch_jtg<J, H, float>(a, which, st);
  return gb ? launch_jtg<J, float, H>(a, which, st) : launch_jtg<J, float, float>(a, which, st);
}

cudaError_t launch(const DeltaArgs &a, Which which, const char *name, cudaStream_t st) {
  cudaError_t e = trace_before(st, name);
  if (e != cudaSuccess) return e;
  e = a.N <= 32 ? launch_j<1>(a, which, st) : a.N <= 64 ? launch_j<2>(a, which, st) : launch_j<4>(a, which, st);
  return e != cudaSuccess ? e : trace_after(st);
}

}  // namespace

cudaError_t launch_delta_steps(const DeltaArgs &a, cudaStream_t st) { return launch(a, kForward, "delta_steps", st); }
cudaError_t launch_delta_steps_save(const DeltaArgs &a, cudaStream_t st) { return launch(a, kForwardSave, "delta_steps_save", st); }
cudaError_t launch_delta_steps_bwd(const DeltaArgs &a, cudaStream_t st) { return launch(a, kBackward, "delta_steps_bwd", st); }

}  // namespace pdssm
