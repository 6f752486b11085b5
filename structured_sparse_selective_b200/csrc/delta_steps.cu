// The gated delta rule step by step (formulas in delta.cuh), forwards and backwards:
// short runs, fp32 inputs with many sequences, and one kernel for a single token.
//
// The columns of H are independent of one another. A column's rows are spread over LPC
// lanes of a warp, in registers for the whole sequence, so k^T H and q^T H are a few sums
// in a lane and log2(LPC) shuffles, and no barrier joins the warps but one every 8 steps.
// A step is one pass over a lane's row pairs,
//   H = a H + u k,  y += q H,  next e: d += k' H   (k' the next step's key),
// four packed instructions a pair (fma.rn.f32x2 works on two rows); the shuffles of y wait
// with those of the next step's d. k and q come from shared memory; loader warps bring
// them there, with v, the decay and beta, in fp32, a tile of 8 steps ahead.
// What bounds it: the chain of steps, each the latency of the sums, the shuffles and one
// update. With a whole column of 32 rows a lane (no shuffles) a step took 460 cycles, with
// eight lanes and four columns a lane 400: eight or sixteen rows a lane keep both the
// issue and the shuffles short. The state moves once in and out.
#include <algorithm>

#include "delta.cuh"

namespace pdssm {

namespace {

constexpr int kTS = 8;  // steps a tile
constexpr int kMaxWarps = 8;     // computing warps of a block
constexpr int kMaxCols = 64;     // their columns
constexpr int kLoaders = 4;      // loader w has the tiles w, w + 4, ...

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

// A loader warp, with every fourth tile. A tile's values wait in registers: fetch() starts
// its loads four tiles ahead, put() writes them to shared memory, so HBM's latency (about
// 1,400 cycles, as long as 9 steps of 32 rows) is behind four tiles' work. The loads are unconditional, from a
// valid place where there is nothing to load: with a branch around each they ran one
// after the other.
template <int J, typename T, typename G>
struct Loader {
  static constexpr int M = kMaxCols / 32;
  const DeltaArgs &a;
  const T *k, *q, *c;
  const G *g, *beta;
  int lane, p0, cols, n;
  int64_t rowk, rowc;
  T kv[kTS][J], qv[kTS][J], cv[kTS][M];
  G gv, bv;
  uint32_t first, step;  // of the places where decays are rounded: the sequence's, and the lane's step

  // `src`: v forwards, dy backwards.
  __device__ Loader(const DeltaArgs &a_, int64_t b, int64_t h, int p0_, int cols_, const void *src)
      : a(a_), lane(threadIdx.x & 31), p0(p0_), cols(cols_), n(0), rowk(a_.Hk * a_.N), rowc(a_.H * a_.P) {
    const int64_t hk = h / (a.H / a.Hk);
    k = static_cast<const T *>(a.k) + b * a.L * rowk + hk * a.N;
    q = static_cast<const T *>(a.q) + b * a.L * rowk + hk * a.N;
    c = static_cast<const T *>(src) + b * a.L * rowc + h * a.P;
    g = static_cast<const G *>(a.g) + b * a.L * a.H + h;
    beta = static_cast<const G *>(a.beta) + b * a.L * a.H + h;
    first = live_steps(a.lengths, b, a.L) > 0 ? (__float_as_uint(to_f32(k[0])) * 2654435769u) ^ __float_as_uint(to_f32(c[0])) : 0;
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
    step = (uint32_t)(t0 + lane);
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
    // A decay's rest is paid in whole steps of the float (2^-24 below 1), in as many of the steps of the sequence as
    // makes their product right: step t rounds at a place of its own in [-1/2, 1/2), t times the golden section, which
    // fills the interval evenly, from a first place by the first key and value, so that short calls one after the other
    // do not all round alike. A decay without a rest stays as it is.
    const float place = (float)((int)((first + step) * 2654435769u) >> 8) * 0x1p-24f;
    const Decay d = decay_of<false>(to_f32(gv));
    if (lane < kTS) tile.ab[lane] = make_float2(fmaf(rintf(fmaf(d.rest, 0x1p24f, place)), 0x1p-24f, d.a), to_f32(bv));
  }
};

// Loader `who` through the tiles: tile i + 1 goes into its buffer while tile i is computed.
template <int J, typename In, typename Fetch>
__device__ __forceinline__ void run_loader(In &in, int who, int64_t tiles, float *smem, int cols, const Fetch &fetch) {
  fetch(who);
  if (who == 0) {
    in.put(Tile<J>(smem, cols, 0));
    fetch(kLoaders);
  }
  __syncthreads();
  for (int64_t i = 0; i < tiles; ++i) {
    if (((i + 1) & (kLoaders - 1)) == who) {
      in.put(Tile<J>(smem, cols, (i + 1) & 1));
      fetch(i + 1 + kLoaders);
    }
    __syncthreads();
  }
}

// How a column's rows lie in LPC lanes: piece j of lane l has rows 4 (LPC j + l) .. + 3.
template <int J>
struct Rows {
  static constexpr int LPC = J == 4 ? 8 : 4, kPieces = 32 * J / (4 * LPC), R = 2 * kPieces;  // R row pairs a lane
  static constexpr int kCols = 32 / LPC;                                                     // columns a warp
};

// The lane's rows of a state column at `p` (null: zeros), row length ld.
template <int J>
__device__ __forceinline__ void load_column(pair2 (&x)[Rows<J>::R], const float *p, int l, int N, int64_t ld, bool in) {
#pragma unroll
  for (int j = 0; j < Rows<J>::kPieces; ++j) {
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int n = 4 * (Rows<J>::LPC * j + l) + r;
      v[r] = p && in && n < N ? p[n * ld] : 0.f;
    }
    x[2 * j] = pack2(v[0], v[1]);
    x[2 * j + 1] = pack2(v[2], v[3]);
  }
}

template <int J>
__device__ __forceinline__ void store_column(const pair2 (&x)[Rows<J>::R], float *p, int l, int N, int64_t ld) {
#pragma unroll
  for (int j = 0; j < Rows<J>::kPieces; ++j) {
    float v[4];
    unpack2(x[2 * j], v[0], v[1]);
    unpack2(x[2 * j + 1], v[2], v[3]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int n = 4 * (Rows<J>::LPC * j + l) + r;
      if (n < N) p[n * ld] = v[r];
    }
  }
}

// The lane's rows of a vector in shared memory.
template <int J>
__device__ __forceinline__ void load_rows(pair2 (&x)[Rows<J>::R], const float *p, int l) {
#pragma unroll
  for (int j = 0; j < Rows<J>::kPieces; ++j) {
    const float4 v = *reinterpret_cast<const float4 *>(p + 4 * (Rows<J>::LPC * j + l));
    x[2 * j] = pack2(v.x, v.y);
    x[2 * j + 1] = pack2(v.z, v.w);
  }
}

__device__ __forceinline__ float total(const pair2 (&s)[2]) {
  float a, b, c, d;
  unpack2(s[0], a, b);
  unpack2(s[1], c, d);
  return (a + c) + (b + d);
}

// One block: the columns p0 ... of head blockIdx.y of sequence blockIdx.z; warps 0 .. warps - 1
// compute, the others load. SAVE: writes e_t and, every a.C steps, the state before them (for
// the backward pass).
template <int J, typename T, typename G, bool SAVE>
__device__ __forceinline__ void forward(const DeltaArgs &a, int group) {
  constexpr int R = Rows<J>::R, LPC = Rows<J>::LPC, kRow = 32 * J;
  extern __shared__ __align__(16) float smem[];
  const int warps = blockDim.x / 32 - kLoaders, warp = threadIdx.x >> 5;
  const int cols = warps * Rows<J>::kCols, p0 = group * cols;
  const int64_t h = blockIdx.y, b = blockIdx.z, bh = b * a.H + h;
  const int64_t len = live_steps(a.lengths, b, a.L);
  if (warp >= warps) {
    Loader<J, T, G> in(a, b, h, p0, cols, a.v);
    run_loader<J>(in, warp - warps, (len + kTS - 1) / kTS, smem, cols, [&](int64_t i) { in.fetch(i * kTS, len - i * kTS); });
    return;
  }
  const int c = threadIdx.x / LPC, l = threadIdx.x % LPC, col = p0 + c, N = (int)a.N;
  const bool in = col < a.P, room = col < a.Pp;
  pair2 st[R], k[R], d[2] = {}, z[2] = {};
  load_column<J>(st, a.h0 ? a.h0 + bh * a.N * a.P + col : nullptr, l, N, a.P, in);
  __syncthreads();
  T *y = static_cast<T *>(a.y) + (b * a.L * a.H + h) * a.P + col;
  float *e_out = SAVE ? a.e + bh * a.L * a.Pp + col : nullptr;
  const int64_t step = SAVE ? a.Pp : a.H * a.P;
  if (len > 0) {
    load_rows<J>(k, Tile<J>(smem, cols, 0).k, l);
#pragma unroll
    for (int r = 0; r < R; ++r) d[r & 1] = fma2(k[r], st[r], r < 2 ? 0 : d[r & 1]);
  }
  const bool writes = l == 0 && (SAVE ? room : in);
  int buf = 0;
  for (int64_t t0 = 0; t0 < len; t0 += kTS, buf ^= 1) {
    const Tile<J> tile(smem, cols, buf), after(smem, cols, buf ^ 1);
    if (SAVE && room && (t0 & (a.C - 1)) == 0)  // a.C is a multiple of kTS
      store_column<J>(st, a.carry + (bh * a.nC + t0 / a.C) * a.N * a.Pp + col, l, N, a.Pp);
    const float *kl = tile.k + 4 * l, *ql = tile.q + 4 * l, *cl = tile.c + c;
    // everything a step reads comes ahead of the shuffles that it waits for
    const auto one = [&](int s, bool last, bool has_y) {
      const float2 ab = tile.ab[s];
      const float v = cl[s * cols];
      pair2 q[R], next[R];
      if (!SAVE) load_rows<J>(q, ql + s * kRow, 0);
      if (last) {  // the next step's key is in the next tile, if there is one
        __syncthreads();
        load_rows<J>(next, after.k, l);
      } else {
        load_rows<J>(next, kl + (s + 1) * kRow, 0);
      }
      float kh = total(d), out = SAVE ? 0.f : total(z);
#pragma unroll
      for (int o = 1; o < LPC; o <<= 1) {
        kh += __shfl_xor_sync(0xffffffffu, kh, o);
        if (!SAVE) out += __shfl_xor_sync(0xffffffffu, out, o);
      }
      const float e = fmaf(-ab.x, kh, v), u = ab.y * e;
      const pair2 aa = pack2(ab.x, ab.x), uu = pack2(u, u);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        st[r] = fma2(k[r], uu, mul2(aa, st[r]));
        d[r & 1] = fma2(next[r], st[r], r < 2 ? 0 : d[r & 1]);
        if (!SAVE) z[r & 1] = fma2(q[r], st[r], r < 2 ? 0 : z[r & 1]);
        k[r] = next[r];
      }
      if (SAVE) {
        if (writes) *e_out = e;
        e_out += step;
      } else if (has_y) {  // the step before's y
        if (writes) st_out(y, out);
        y += step;
      }
    };
    if (len - t0 >= kTS) {
      one(0, false, t0 > 0);
#pragma unroll
      for (int s = 1; s < kTS; ++s) one(s, s == kTS - 1, true);
    } else {
      const int n = (int)(len - t0);
      for (int s = 0; s < n; ++s) one(s, s + 1 == n, t0 + s > 0);
    }
  }
  if (SAVE) return;
  if (len > 0) {
    float out = total(z);
#pragma unroll
    for (int o = 1; o < LPC; o <<= 1) out += __shfl_xor_sync(0xffffffffu, out, o);
    if (l == 0 && in) st_out(y, out);
    y += step;
  }
  if (!in) return;
  for (int64_t t = len + l; t < a.L; t += LPC) st_out(y + (t - len) * step, 0.f);
  if (a.h_final) store_column<J>(st, a.h_final + bh * a.N * a.P + col, l, N, a.P);
}

// The adjoint X runs from the last step to the first; writes dv_t, du_t, X at the end
// of each chunk of a.C steps, and dh0. A step is
//   X += dy q,  du = k X (sums and shuffles),  X = a (X - w k).
template <int J, typename T, typename G>
__device__ __forceinline__ void backward(const DeltaArgs &a, int group) {
  constexpr int R = Rows<J>::R, LPC = Rows<J>::LPC, kRow = 32 * J;
  extern __shared__ __align__(16) float smem[];
  const int warps = blockDim.x / 32 - kLoaders, warp = threadIdx.x >> 5;
  const int cols = warps * Rows<J>::kCols, p0 = group * cols;
  const int64_t h = blockIdx.y, b = blockIdx.z, bh = b * a.H + h;
  const int64_t len = live_steps(a.lengths, b, a.L);
  const int64_t tiles = (len + kTS - 1) / kTS;
  if (warp >= warps) {
    Loader<J, T, G> in(a, b, h, p0, cols, a.dy);
    run_loader<J>(in, warp - warps, tiles, smem, cols, [&](int64_t i) {  // tiles from the last to the first
      const int64_t t0 = (tiles - 1 - i) * kTS;
      in.fetch(t0, i < tiles ? len - t0 : 0);
    });
    return;
  }
  const int c = threadIdx.x / LPC, l = threadIdx.x % LPC, col = p0 + c, N = (int)a.N;
  const bool in = col < a.P, room = col < a.Pp;
  pair2 x[R];
  load_column<J>(x, a.dh_final ? a.dh_final + bh * a.N * a.P + col : nullptr, l, N, a.P, in);
  __syncthreads();
  T *dv = static_cast<T *>(a.dv) + (b * a.L * a.H + h) * a.P + col;
  float *du_out = a.du + bh * a.L * a.Pp + col;
  pair2 k[R], q[R];
  if (tiles > 0) {
    const Tile<J> tile(smem, cols, 0);
    const int s = (int)(len - (tiles - 1) * kTS) - 1;
    load_rows<J>(k, tile.k + s * kRow, l);
    load_rows<J>(q, tile.q + s * kRow, l);
  }
  const bool writes_du = l == 0 && room, writes_dv = l == 0 && in;
  const int64_t step_du = a.Pp, step_dv = a.H * a.P;
  T *dv_at = dv + (len - 1) * step_dv;
  du_out += (len - 1) * step_du;
  int buf = 0;
  for (int64_t i = 0; i < tiles; ++i, buf ^= 1) {
    const int64_t t0 = (tiles - 1 - i) * kTS;
    const Tile<J> tile(smem, cols, buf), before(smem, cols, buf ^ 1);
    if (room && (i == 0 || ((t0 + kTS) & (a.C - 1)) == 0))  // a.C is a multiple of kTS
      store_column<J>(x, a.xcarry + (bh * a.nC + t0 / a.C) * a.N * a.Pp + col, l, N, a.Pp);
    const float *kl = tile.k + 4 * l, *ql = tile.q + 4 * l, *cl = tile.c + c;
    const auto one = [&](int s) {
      const float2 ab = tile.ab[s];
      const float dy = cl[s * cols];
      // the key and query of the step before, ahead of the shuffles
      pair2 kn[R], qn[R];
      if (s == 0) {  // it is in the tile before, if there is one
        __syncthreads();
        load_rows<J>(kn, before.k + (kTS - 1) * kRow, l);
        load_rows<J>(qn, before.q + (kTS - 1) * kRow, l);
      } else {
        load_rows<J>(kn, kl + (s - 1) * kRow, 0);
        load_rows<J>(qn, ql + (s - 1) * kRow, 0);
      }
      const pair2 dd = pack2(dy, dy), aa = pack2(ab.x, ab.x);
      pair2 sum[2];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        x[r] = fma2(q[r], dd, x[r]);
        sum[r & 1] = fma2(k[r], x[r], r < 2 ? 0 : sum[r & 1]);
      }
      float du = total(sum);
#pragma unroll
      for (int o = 1; o < LPC; o <<= 1) du += __shfl_xor_sync(0xffffffffu, du, o);
      const float w = ab.y * du;
      const pair2 ww = pack2(-w, -w);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        x[r] = mul2(aa, fma2(k[r], ww, x[r]));
        k[r] = kn[r];
        q[r] = qn[r];
      }
      if (writes_du) *du_out = du;
      if (writes_dv) st_out(dv_at, w);
      du_out -= step_du;
      dv_at -= step_dv;
    };
    const int64_t n = len - t0;
    if (n >= kTS) {
#pragma unroll
      for (int s = kTS - 1; s >= 0; --s) one(s);
    } else {
      for (int s = (int)n - 1; s >= 0; --s) one(s);
    }
  }
  if (!in) return;
  for (int64_t t = len + l; t < a.L; t += LPC) st_out(dv + t * a.H * a.P, 0.f);
  if (a.dh0) store_column<J>(x, a.dh0 + bh * a.N * a.P + col, l, N, a.P);
}

// Nothing here waits for another role: the error word of a workspace, if there is one, says so.
__device__ __forceinline__ void clear_error(const DeltaArgs &a) {
  if (a.err && threadIdx.x + blockIdx.x + blockIdx.y + blockIdx.z == 0) *a.err = 0;
}

// grid: (column groups, heads, batch)
template <int J, typename T, typename G>
__global__ void __launch_bounds__(32 * (kMaxWarps + kLoaders)) delta_steps_kernel(DeltaArgs a) {
  clear_error(a);
  forward<J, T, G, false>(a, blockIdx.x);
}

// The states and the adjoints of a backward pass do not need one another: their blocks take
// turns, so that few sequences fill more SMs. grid: (2 x column groups, heads, batch)
template <int J, typename T, typename G>
__global__ void __launch_bounds__(32 * (kMaxWarps + kLoaders)) delta_steps_both_kernel(DeltaArgs a) {
  clear_error(a);
  if (blockIdx.x & 1) backward<J, T, G>(a, blockIdx.x >> 1);
  else forward<J, T, G, true>(a, blockIdx.x >> 1);
}

// ------------------------------------------------------------------ one token

// One step of every sequence: the state is read and written once and that is the cost, so
// the rows are spread over the lanes for wide loads: lane (rg, cl) = (lane / 4, lane % 4)
// has columns 4 cl .. + 3 of the warp's 16 and rows 32 j + 4 rg .. + 3. The warps are on
// their own; k^T H and q^T H are finished by three shuffles.
template <int J, typename T, typename G>
__global__ void __launch_bounds__(128) delta_token_kernel(DeltaArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rg = lane >> 2;
  const int col = (blockIdx.x * (blockDim.x >> 5) + warp) * 16 + 4 * (lane & 3);
  const int64_t h = blockIdx.y, b = blockIdx.z, bh = b * a.H + h, hk = h / (a.H / a.Hk);
  const int N = (int)a.N, P = (int)a.P;
  const bool on = !a.lengths || a.lengths[b] > 0;
  const float *h0 = a.h0 ? a.h0 + bh * N * P : nullptr;
  float *hf = a.h_final ? a.h_final + bh * N * P : nullptr;
  const bool wide = P % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.h0) | reinterpret_cast<uintptr_t>(a.h_final)) & 15) == 0;
  // loads come from a valid place where there is nothing, without a branch around each
  float st[4 * J][4];
  const auto row = [&](int i) { return 32 * (i / 4) + 4 * rg + (i & 3); };
  if (h0 && wide) {
#pragma unroll
    for (int i = 0; i < 4 * J; ++i) {
      const float4 x = *reinterpret_cast<const float4 *>(h0 + min(row(i), N - 1) * P + min(col, P - 4));
      st[i][0] = x.x; st[i][1] = x.y; st[i][2] = x.z; st[i][3] = x.w;
    }
  } else if (h0) {
#pragma unroll
    for (int i = 0; i < 4 * J; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) st[i][c] = h0[min(row(i), N - 1) * P + min(col + c, P - 1)];
  } else {
#pragma unroll
    for (int i = 0; i < 4 * J; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) st[i][c] = 0.f;
  }
  float k[4 * J], q[4 * J], v[4] = {}, y[4] = {};
  float beta = 0.f;
  if (on) {
    const T *kp = static_cast<const T *>(a.k) + (b * a.Hk + hk) * N, *qp = static_cast<const T *>(a.q) + (b * a.Hk + hk) * N;
#pragma unroll
    for (int i = 0; i < 4 * J; ++i) {
      k[i] = ldf(kp + min(row(i), N - 1));
      q[i] = ldf(qp + min(row(i), N - 1));
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = ldf(static_cast<const T *>(a.v) + bh * P + min(col + c, P - 1));
    const Decay decay = decay_of<true>(ldf(static_cast<const G *>(a.g) + bh));
    beta = ldf(static_cast<const G *>(a.beta) + bh);
#pragma unroll
    for (int i = 0; i < 4 * J; ++i) {
      k[i] = row(i) < N ? k[i] : 0.f;
      q[i] = row(i) < N ? q[i] * a.scale : 0.f;
    }
    float d[4] = {};
#pragma unroll
    for (int i = 0; i < 4 * J; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) d[c] = fmaf(k[i], st[i][c], d[c]);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1)
#pragma unroll
      for (int c = 0; c < 4; ++c) d[c] += __shfl_xor_sync(0xffffffffu, d[c], o);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float u = beta * fmaf(-decay.a, d[c], v[c]);
#pragma unroll
      for (int i = 0; i < 4 * J; ++i) {
        st[i][c] = fmaf(k[i], u, fmaf(decay.a, st[i][c], decay.rest * st[i][c]));
        y[c] = fmaf(q[i], st[i][c], y[c]);
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1)
#pragma unroll
      for (int c = 0; c < 4; ++c) y[c] += __shfl_xor_sync(0xffffffffu, y[c], o);
  }
  clear_error(a);  // here, where nothing waits for it any more
  if (rg == 0) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (col + c < P) st_out(static_cast<T *>(a.y) + bh * P + col + c, y[c]);
  }
  if (!hf) return;
#pragma unroll
  for (int i = 0; i < 4 * J; ++i) {
    const int n = row(i);
    if (n >= N) continue;
    float *p = hf + n * P + col;
    if (wide) {
      if (col < P) *reinterpret_cast<float4 *>(p) = make_float4(st[i][0], st[i][1], st[i][2], st[i][3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (col + c < P) p[c] = st[i][c];
    }
  }
}

enum Which { kForward, kBoth, kToken };

template <int J, typename T, typename G>
cudaError_t launch_jtg(const DeltaArgs &a, Which which, cudaStream_t st) {
  if (which == kToken) {
    const int groups = (int)((a.P + 15) / 16), warps = std::min(groups, 4);
    delta_token_kernel<J, T, G><<<dim3((unsigned)((groups + warps - 1) / warps), (unsigned)a.H, (unsigned)a.Bt), 32 * warps, 0, st>>>(a);
    return cudaGetLastError();
  }
  // up to 8 warps share a block's loaded tiles; with few sequences the columns are spread
  // over more blocks, down to 2 warps, until there is one an SM
  constexpr int kCols = Rows<J>::kCols;
  const int all = (int)((a.P + kCols - 1) / kCols);
  int warps = std::min(all, kMaxWarps);
  while (warps > 2 && a.Bt * a.H * ((all + warps - 1) / warps) < 148) warps = (warps + 1) / 2;
  const dim3 grid((unsigned)((all + warps - 1) / warps) * (which == kBoth ? 2 : 1), (unsigned)a.H, (unsigned)a.Bt);
  const size_t smem = Tile<J>::bytes(warps * kCols);
  auto kern = which == kForward ? delta_steps_kernel<J, T, G> : delta_steps_both_kernel<J, T, G>;
  kern<<<grid, 32 * (warps + kLoaders), smem, st>>>(a);
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

cudaError_t launch_delta_steps(const DeltaArgs &a, cudaStream_t st) {
  return a.L == 1 ? launch(a, kToken, "delta_token", st) : launch(a, kForward, "delta_steps", st);
}
cudaError_t launch_delta_steps_both(const DeltaArgs &a, cudaStream_t st) { return launch(a, kBoth, "delta_steps_both", st); }

}  // namespace pdssm
