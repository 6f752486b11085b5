// The norm of every query and key head with the position rotation in the same
// pass, forward and backward.
//
// For one head x (N values) of one token, with w the weight (1 when absent):
//   r = 1 / sqrt(share * sum_i x_i^2 + eps),  share = 1/N (RMS) or 1 (L2)
//   z = x r w;  y = z with its first `rot` values turned pair by pair by the
//   token's angles position * inv_freq[i], i < rot/2
// and backwards, with d = dy turned by the negative angles:
//   dw += d x r;  dx = r (d w - x r * share * sum_i d_i w_i x_i r)
//
// What bounds it: HBM and the issue rate, both near. Each value is read once and written
// once (backward: x and dy read, dx written). A head is held by a group of 2^g lanes, two
// pieces of four or eight values a lane: a piece of the first rotated half and its partner in the
// second, so a pair turns inside a lane (with one 16-byte piece a lane and the partner by
// shuffles the LM layer took 80 us, issue-bound). Heads whose size, rotated width or
// alignment do not allow pieces take the one-value-a-lane path with the partner read
// through shared memory.
// The angles are the same for all heads of a token: a block computes them once for
// its tile of tokens. Their product and reduction to [-pi, pi] are in double
// precision, since at position 10^6 a float's angle is off by 0.03.
#include <algorithm>

#include "launch.h"

namespace pdssm {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 8;   // tokens a tile
// Blocks of 256 threads of q and of k each: together four an SM, three backwards, which
// needs the registers.
constexpr int blocks_of(bool bwd) { return bwd ? 148 * 3 / 2 : 148 * 2; }

enum Turn { kNone, kHalves, kNeighbours };

// V values moved as one access: 4 floats, 4 or 8 bf16.
template <int V>
__device__ __forceinline__ void load(const float *p, float *v) {
  static_assert(V == 4, "16 bytes");
  const float4 x = *reinterpret_cast<const float4 *>(p);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
}
template <int V>
__device__ __forceinline__ void load(const __nv_bfloat16 *p, float *v) {
  uint32_t w[V / 2];
  if constexpr (V == 8) {
    const uint4 x = *reinterpret_cast<const uint4 *>(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    w[0] = x.x; w[1] = x.y;
  }
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <int V>
__device__ __forceinline__ void store(float *p, const float *v) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) {
  uint32_t w[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  if constexpr (V == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// cos and sin of position * f, the product reduced by whole turns in double.
// `coarse`: by the hardware's sine and cosine, off by up to 2^-21 (results rounded to bf16).
__device__ __forceinline__ float2 angle(int position, float f, bool coarse) {
  const double a = (double)position * (double)f;
  const double turns = rint(a * 0.15915494309189535);
  double r = fma(turns, -6.283185307179586, a);
  r = fma(turns, -2.4492935982947064e-16, r);
  float s, c;
  if (coarse) __sincosf((float)r, &s, &c);
  else sincosf((float)r, &s, &c);
  return make_float2(c, s);
}

struct Args {
  int64_t rows;     // batch * seqlen
  int64_t seqlen;
  int heads[2];     // of q, of k
  int N, rot, interleaved, tile;
  float share, eps;
  const void *x[2], *dy[2];
  void *out[2];     // y forward, dx backward
  const float *w[2], *inv_freq;
  const int *positions;  // [rows] or null: the token's place in its sequence
  float *part[2];   // backward with weights: [gridDim.x][N] partial sums of dw
};

// The angles of tokens [t0, t0 + nt) into tab[token][rot / 2].
__device__ __forceinline__ void fill_angles(const Args &a, int64_t t0, int nt, float2 *tab, bool coarse) {
  const int h = a.rot / 2;
  for (int i = threadIdx.x; i < nt * h; i += kThreads) {
    const int t = i / h, j = i - t * h;
    const int64_t row = t0 + t;
    const int pos = a.positions ? a.positions[row] : (int)(row % a.seqlen);
    tab[i] = angle(pos, a.inv_freq[j], coarse);
  }
}

// 1 / sqrt(s): the hardware's, one Newton step nearer (without it, a head of one value, whose
// gradient is a difference of nearly equal terms, is off by more than fp32's rounding).
__device__ __forceinline__ float inverse_sqrt(float s) {
  const float r = rsqrtf(s), e = fmaf(-s * r, r, 1.f);
  return s > 0.f && s < INFINITY ? fmaf(0.5f * r, e, r) : r;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float s) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Turns the lane's two pieces, values [ia, ia + V) and [ib, ib + V) of the head, by the
// token's angles; `sign` -1 turns back.
template <int V, int TURN>
__device__ __forceinline__ void turn_pieces(float (&v)[2 * V], int ia, int ib, int rot, const float2 *tab, float sign) {
  const auto pair = [&](float &x, float &y, float c, float s) {
    const float p = x, q = y;
    s *= sign;
    x = p * c - q * s;
    y = q * c + p * s;
  };
  if (TURN == kHalves) {
    if (ia < rot) {  // then the second piece is the first's partner
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        const float4 t = *reinterpret_cast<const float4 *>(tab + ia + e);
        pair(v[e], v[V + e], t.x, t.y);
        pair(v[e + 1], v[V + e + 1], t.z, t.w);
      }
    }
  } else if (TURN == kNeighbours) {
#pragma unroll
    for (int e = 0; e < 2 * V; e += 2) {
      const int i = e < V ? ia + e : ib + e - V;
      if (i < rot) pair(v[e], v[e + 1], tab[i >> 1].x, tab[i >> 1].y);
    }
  }
}

// LANES lanes hold one head, two pieces of V values a lane (FULL: all lanes do);
// blockIdx.y: 0 = q, 1 = k. U heads of a lane group are in flight at once, so that their
// loads cover HBM's latency.
template <typename T, int V, int LANES, int TURN, bool BWD, bool FULL>
__global__ void __launch_bounds__(kThreads, BWD ? 3 : 4) qk_piece_kernel(Args a) {
  extern __shared__ __align__(16) float2 tab[];
  constexpr int U = V == 8 ? 2 : BWD ? 2 : 4, kGroups = kThreads / LANES;
  const int which = blockIdx.y, H = a.heads[which], N = a.N, half = a.rot / 2;
  const int group = threadIdx.x / LANES, gl = threadIdx.x % LANES;
  // the lane's pieces: partners first, then what does not turn
  const int pairs = TURN == kHalves ? half / V : 0;
  const int ia = gl < pairs ? V * gl : V * (2 * gl), ib = gl < pairs ? ia + half : ia + V;
  const bool ina = FULL || ia < N, inb = FULL || ib < N;
  const unsigned per_head = H > 1 ? 0xffffffffu / (unsigned)H + 1 : 0;  // item / H as a product (items < 2^16)
  float wv[2 * V], dw[BWD ? 2 * V : 1];
#pragma unroll
  for (int e = 0; e < 2 * V; ++e) {
    const int i = e < V ? ia + e : ib + e - V;
    wv[e] = a.w[which] && i < N ? a.w[which][i] : 1.f;
    if (BWD) dw[e] = 0.f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * a.tile; t0 < a.rows; t0 += (int64_t)gridDim.x * a.tile) {
    const int nt = (int)(a.rows - t0 < a.tile ? a.rows - t0 : a.tile);
    if (TURN != kNone) {
      __syncthreads();
      fill_angles(a, t0, nt, tab, sizeof(T) == 2);
      __syncthreads();
    }
    const int items = nt * H;
    const T *x = static_cast<const T *>(a.x[which]) + t0 * H * N;
    const T *dy = static_cast<const T *>(a.dy[which]) + (BWD ? t0 * H * N : 0);
    T *out = static_cast<T *>(a.out[which]) + t0 * H * N;
    // `whole`: every group of the block has a head in each of the U places
    const auto batch = [&](int it0, bool whole) {
      float v[U][2 * V], d[BWD ? U : 1][2 * V];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int it = it0 + u * kGroups + group;
        if (!(FULL && whole)) {
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {
            v[u][e] = 0.f;
            if (BWD) d[BWD ? u : 0][e] = 0.f;
          }
        }
        if (whole || it < items) {
          if (ina) load<V>(x + it * N + ia, v[u]);
          if (inb) load<V>(x + it * N + ib, v[u] + V);
          if (BWD && ina) load<V>(dy + it * N + ia, d[BWD ? u : 0]);
          if (BWD && inb) load<V>(dy + it * N + ib, d[BWD ? u : 0] + V);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!whole && it0 + u * kGroups >= items) break;  // the same for all: shuffles follow
        const int it = it0 + u * kGroups + group;
        const bool la = (whole || it < items) && ina, lb = (whole || it < items) && inb;
        const int token = TURN != kNone && (whole || it < items) ? (H > 1 ? (int)__umulhi((unsigned)it, per_head) : it) : 0;
        const float2 *row = tab + token * half;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int e = 0; e < 2 * V; e += 2) {
          s0 = fmaf(v[u][e], v[u][e], s0);
          s1 = fmaf(v[u][e + 1], v[u][e + 1], s1);
        }
        const float r = inverse_sqrt(fmaf(group_sum<LANES>(s0 + s1), a.share, a.eps));
        if (!BWD) {
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) v[u][e] = v[u][e] * r * wv[e];
          turn_pieces<V, TURN>(v[u], ia, ib, a.rot, row, 1.f);
          if (la) store<V>(out + it * N + ia, v[u]);
          if (lb) store<V>(out + it * N + ib, v[u] + V);
        } else {
          float(&g)[2 * V] = d[BWD ? u : 0];
          turn_pieces<V, TURN>(g, ia, ib, a.rot, row, -1.f);
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) {  // r may be infinite where there is nothing
            const float xh = (e < V ? la : lb) ? v[u][e] * r : 0.f;
            dw[BWD ? e : 0] = fmaf(g[e], xh, dw[BWD ? e : 0]);
            g[e] *= wv[e];
            v[u][e] = xh;
            dot = fmaf(g[e], xh, dot);
          }
          dot = group_sum<LANES>(dot) * a.share;
#pragma unroll
          for (int e = 0; e < 2 * V; ++e) g[e] = r * (g[e] - v[u][e] * dot);
          if (la) store<V>(out + it * N + ia, g);
          if (lb) store<V>(out + it * N + ib, g + V);
        }
      }
    };
    int it0 = 0;
    for (; it0 + kGroups * U <= items; it0 += kGroups * U) batch(it0, true);
    if (it0 < items) batch(it0, false);
  }
  if (BWD && a.part[which]) {
    // the block's share of dw: lane groups added in a fixed order
    __shared__ float acc[BWD ? kGroups : 1][2 * V * LANES + 1];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) {
      const int i = e < V ? ia + e : ib + e - V;
      if (i < N) acc[group][i] = dw[BWD ? e : 0];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < N; i += kThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int g = 0; g < kGroups; ++g) s += acc[g][i];
      a.part[which][(int64_t)blockIdx.x * N + i] = s;
    }
  }
}

// One warp a head, value lane + 32 e in slot e: any N <= 128, any rotated width,
// any alignment. The rotation's partner comes from the warp's row in shared memory.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_value_kernel(Args a) {
  extern __shared__ float2 tab[];
  constexpr int E = PDSSM_MAX_N / 32, kWarps = kThreads / 32;
  __shared__ float buf[kWarps][PDSSM_MAX_N];
  const int which = blockIdx.y, H = a.heads[which];
  const T *x = static_cast<const T *>(a.x[which]);
  const T *dy = static_cast<const T *>(a.dy[which]);
  T *out = static_cast<T *>(a.out[which]);
  const float *w = a.w[which];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = a.rot / 2;
  float wv[E], dw[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = lane + 32 * e;
    wv[e] = (w && i < a.N) ? w[i] : 1.f;
    dw[e] = 0.f;
  }
  auto turn = [&](float *v, const float2 *row, float sign) {
    __syncwarp();
#pragma unroll
    for (int e = 0; e < E; ++e) buf[warp][lane + 32 * e] = v[e];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = lane + 32 * e;
      if (i < a.rot) {
        const bool low = a.interleaved ? !(i & 1) : i < half;
        const int j = a.interleaved ? (i ^ 1) : (low ? i + half : i - half);
        const float2 cs = row[a.interleaved ? i >> 1 : (low ? i : j)];
        const float s = sign * cs.y, o = buf[warp][j];
        v[e] = low ? v[e] * cs.x - o * s : v[e] * cs.x + o * s;
      }
    }
  };
  for (int64_t t0 = (int64_t)blockIdx.x * a.tile; t0 < a.rows; t0 += (int64_t)gridDim.x * a.tile) {
    const int nt = (int)(a.rows - t0 < a.tile ? a.rows - t0 : a.tile);
    if (half) {
      __syncthreads();
      fill_angles(a, t0, nt, tab, sizeof(T) == 2);
      __syncthreads();
    }
    for (int it = warp; it < nt * H; it += kWarps) {
      const int64_t at = (t0 * H + it) * a.N;
      const float2 *row = tab + (it / H) * half;
      float v[E], d[E], s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = lane + 32 * e;
        v[e] = i < a.N ? ldf(x + at + i) : 0.f;
        d[e] = (BWD && i < a.N) ? ldf(dy + at + i) : 0.f;
        s = fmaf(v[e], v[e], s);
      }
      const float r = inverse_sqrt(fmaf(group_sum<32>(s), a.share, a.eps));
      if (!BWD) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = v[e] * r * wv[e];
        if (half) turn(v, row, 1.f);
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (lane + 32 * e < a.N) st_out(out + at + lane + 32 * e, v[e]);
      } else {
        if (half) turn(d, row, -1.f);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (lane + 32 * e < a.N) {
            const float xh = v[e] * r;
            dw[e] = fmaf(d[e], xh, dw[e]);
            d[e] *= wv[e];
            v[e] = xh;
            dot = fmaf(d[e], xh, dot);
          }
        }
        dot = group_sum<32>(dot) * a.share;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (lane + 32 * e < a.N) st_out(out + at + lane + 32 * e, r * (d[e] - v[e] * dot));
      }
    }
  }
  if (BWD && a.part[which]) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) buf[warp][lane + 32 * e] = dw[e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.N; i += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < kWarps; ++g) s += buf[g][i];
      a.part[which][(int64_t)blockIdx.x * a.N + i] = s;
    }
  }
}

// dw[i] = the blocks' shares in a fixed order, in double: 32 slices of the blocks side by
// side, then the slices. A block has 32 values of q's (blockIdx.y 0) or k's weight.
__global__ void __launch_bounds__(1024) qk_weight_kernel(const float *pq, const float *pk, int nblk, int N, float *dwq,
                                                         float *dwk) {
  const float *p = blockIdx.y ? pk : pq;
  float *dw = blockIdx.y ? dwk : dwq;
  if (!p || !dw) return;
  __shared__ double acc[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  double s = 0;
  if (i < N)
#pragma unroll 10
    for (int b = slice; b < nblk; b += 32) s += p[(int64_t)b * N + i];
  acc[slice][lane] = s;
  __syncthreads();
  if (slice == 0 && i < N) {
    double t = 0;
#pragma unroll 8
    for (int k = 0; k < 32; ++k) t += acc[k][lane];
    dw[i] = (float)t;
  }
}

template <typename T, int V, int LANES, int TURN, bool BWD>
void launch_full(const Args &a, dim3 grid, size_t smem, cudaStream_t st) {
  if (a.N == 2 * V * LANES) qk_piece_kernel<T, V, LANES, TURN, BWD, true><<<grid, kThreads, smem, st>>>(a);
  else qk_piece_kernel<T, V, LANES, TURN, BWD, false><<<grid, kThreads, smem, st>>>(a);
}

template <typename T, int V, int TURN, bool BWD>
void launch_lanes(const Args &a, dim3 grid, size_t smem, cudaStream_t st) {
  const int lanes = (a.N / V + 1) / 2;
  if (lanes <= 4) launch_full<T, V, 4, TURN, BWD>(a, grid, smem, st);
  else if (V == 8 || lanes <= 8) launch_full<T, V, 8, TURN, BWD>(a, grid, smem, st);
  else if constexpr (V == 4) launch_full<T, V, 16, TURN, BWD>(a, grid, smem, st);
}

template <typename T, int V, bool BWD>
void launch_turn(const Args &a, dim3 grid, size_t smem, cudaStream_t st) {
  if (!a.rot) launch_lanes<T, V, kNone, BWD>(a, grid, smem, st);
  else if (a.interleaved) launch_lanes<T, V, kNeighbours, BWD>(a, grid, smem, st);
  else launch_lanes<T, V, kHalves, BWD>(a, grid, smem, st);
}

// Whether heads can be moved in pieces of `v` values, which a pair may not cross, of `size` bytes each.
bool pieces_fit(const Args &a, int v, int size, bool bwd) {
  uintptr_t all = 0;
  for (int i = 0; i < 2; ++i)
    all |= reinterpret_cast<uintptr_t>(a.x[i]) | reinterpret_cast<uintptr_t>(a.out[i]) | (bwd ? reinterpret_cast<uintptr_t>(a.dy[i]) : 0);
  return a.N % v == 0 && all % (v * size) == 0 && (!a.rot || a.interleaved || a.rot % (2 * v) == 0);
}

template <bool BWD>
cudaError_t launch(const Args &a, int io_t, int blocks, cudaStream_t st) {
  const dim3 grid(blocks, 2);
  const size_t smem = sizeof(float2) * a.tile * (a.rot / 2);
  using B = __nv_bfloat16;
  if (io_t == PDSSM_BF16) {
    // sixteen values a lane where registers allow it (forwards): fewer lanes to sum over and half the accesses
    if (!BWD && pieces_fit(a, 8, 2, BWD)) {
      if constexpr (!BWD) launch_turn<B, 8, BWD>(a, grid, smem, st);
    } else if (pieces_fit(a, 4, 2, BWD)) {
      launch_turn<B, 4, BWD>(a, grid, smem, st);
    } else {
      qk_value_kernel<B, BWD><<<grid, kThreads, smem, st>>>(a);
    }
  } else if (pieces_fit(a, 4, 4, BWD)) {
    launch_turn<float, 4, BWD>(a, grid, smem, st);
  } else {
    qk_value_kernel<float, BWD><<<grid, kThreads, smem, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

// Tokens a tile: up to 8 share one table of angles and one pair of barriers, fewer
// when that would leave SMs without a block.
static int qk_tile(int64_t rows, bool bwd) {
  return (int)std::min<int64_t>(kMaxTile, std::max<int64_t>(1, rows / blocks_of(bwd)));
}

static int qk_blocks(int64_t rows, bool bwd) {
  const int64_t tiles = (rows + qk_tile(rows, bwd) - 1) / qk_tile(rows, bwd);
  return (int)std::min<int64_t>(tiles, blocks_of(bwd));
}

int qk_norm_bwd_blocks(int64_t rows) { return qk_blocks(rows, true); }

cudaError_t launch_qk_norm(const QkNormArgs &q, bool bwd, cudaStream_t st) {
  Args a{};
  a.rows = q.rows; a.seqlen = q.seqlen;
  a.N = (int)q.N; a.rot = q.rot; a.interleaved = q.interleaved;
  // items of a tile are counted in 16 bits
  a.tile = std::max(q.heads[0], q.heads[1]) > 4096 ? 1 : qk_tile(q.rows, bwd);
  a.share = q.l2 ? 1.f : 1.f / (float)q.N;
  a.eps = q.eps;
  a.inv_freq = q.inv_freq; a.positions = q.positions;
  const int blocks = qk_blocks(q.rows, bwd);
  for (int i = 0; i < 2; ++i) {
    a.heads[i] = (int)q.heads[i]; a.x[i] = q.x[i]; a.dy[i] = q.dy[i]; a.out[i] = q.out[i]; a.w[i] = q.w[i];
    a.part[i] = (bwd && q.dw[i]) ? q.part + (int64_t)i * blocks * q.N : nullptr;
  }
  cudaError_t e = trace_before(st, bwd ? "qk_norm_bwd" : "qk_norm");
  if (e != cudaSuccess) return e;
  e = bwd ? launch<true>(a, q.io_t, blocks, st) : launch<false>(a, q.io_t, blocks, st);
  if (e != cudaSuccess) return e;
  if ((e = trace_after(st)) != cudaSuccess) return e;
  if (bwd && (q.dw[0] || q.dw[1])) {
    if ((e = trace_before(st, "qk_weight_grad")) != cudaSuccess) return e;
    qk_weight_kernel<<<dim3((a.N + 31) / 32, 2), 1024, 0, st>>>(a.part[0], a.part[1], blocks, a.N, q.dw[0], q.dw[1]);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = trace_after(st);
  }
  return e;
}

}  // namespace pdssm
