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
// What bounds it: HBM. Each value is read once and written once (backward: x and
// dy read, dx written); the arithmetic is a few operations a value. A head is held
// by a group of 2^g lanes in 16-byte (or 8-byte) pieces, so the sum is a shuffle
// reduction inside the group and a pair's partner is in the same lane or a fixed
// number of lanes away; heads whose size, rotated width or alignment do not allow
// that take the one-value-a-lane path with the partner read through shared memory.
// The angles are the same for all heads of a token: a block computes them once for
// its tile of tokens. Their product and reduction to [-pi, pi] are in double
// precision, since at position 10^6 a float's angle is off by 0.03.
#include <algorithm>

#include "launch.h"

namespace pdssm {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 8;   // tokens a tile
constexpr int kUnroll = 4;    // heads in flight per lane group

template <typename T, int VEC>
struct Piece;  // VEC values moved as one access
template <>
struct Piece<float, 4> { using V = float4; };
template <>
struct Piece<float, 2> { using V = float2; };
template <>
struct Piece<float, 1> { using V = float; };
template <>
struct Piece<__nv_bfloat16, 8> { using V = uint4; };
template <>
struct Piece<__nv_bfloat16, 4> { using V = uint2; };
template <>
struct Piece<__nv_bfloat16, 1> { using V = __nv_bfloat16; };

template <typename T, int VEC>
__device__ __forceinline__ void load_piece(const T *p, float *v) {
  union { typename Piece<T, VEC>::V raw; T e[VEC]; } u;
  u.raw = *reinterpret_cast<const typename Piece<T, VEC>::V *>(p);
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = to_f32(u.e[i]);
}

__device__ __forceinline__ void put(float &o, float v) { o = v; }
__device__ __forceinline__ void put(__nv_bfloat16 &o, float v) { o = __float2bfloat16_rn(v); }

template <typename T, int VEC>
__device__ __forceinline__ void store_piece(T *p, const float *v) {
  union U { typename Piece<T, VEC>::V raw; T e[VEC]; __device__ U() {} } u;
#pragma unroll
  for (int i = 0; i < VEC; ++i) put(u.e[i], v[i]);
  *reinterpret_cast<typename Piece<T, VEC>::V *>(p) = u.raw;
}

// cos and sin of position * f, the product reduced by whole turns in double.
__device__ __forceinline__ float2 angle(int position, float f) {
  const double a = (double)position * (double)f;
  const double turns = rint(a * 0.15915494309189535);
  double r = fma(turns, -6.283185307179586, a);
  r = fma(turns, -2.4492935982947064e-16, r);
  float s, c;
  sincosf((float)r, &s, &c);
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
__device__ __forceinline__ void fill_angles(const Args &a, int64_t t0, int nt, float2 *tab) {
  const int h = a.rot / 2;
  for (int i = threadIdx.x; i < nt * h; i += kThreads) {
    const int t = i / h, j = i - t * h;
    const int64_t row = t0 + t;
    const int pos = a.positions ? a.positions[row] : (int)(row % a.seqlen);
    tab[i] = angle(pos, a.inv_freq[j]);
  }
}

// Turns the lane's piece. Values [i0, i0 + VEC) of the head; `sign` -1 turns back.
// VEC > 1: partners are in the lane (interleaved) or rot / 2 / VEC lanes away.
template <int VEC, int LANES>
__device__ __forceinline__ void turn_piece(float *v, int i0, const Args &a, const float2 *tab, float sign) {
  const int h = a.rot / 2;
  if (a.interleaved) {
    if (i0 < a.rot) {
#pragma unroll
      for (int e = 0; e + 1 < VEC; e += 2) {
        if (i0 + e < a.rot) {
          const float2 cs = tab[(i0 + e) >> 1];
          const float s = sign * cs.y, p = v[e], q = v[e + 1];
          v[e] = p * cs.x - q * s;
          v[e + 1] = q * cs.x + p * s;
        }
      }
    }
  } else {
    const bool low = i0 < h, in = i0 < a.rot;
    const int lane = threadIdx.x & 31, away = h / VEC;
    const int src = !in ? lane : low ? lane + away : lane - away;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float o = __shfl_sync(0xffffffffu, v[e], src);
      if (in) {
        const float2 cs = tab[low ? i0 + e : i0 + e - h];
        const float s = sign * cs.y;
        v[e] = low ? v[e] * cs.x - o * s : v[e] * cs.x + o * s;
      }
    }
  }
}

template <int LANES>
__device__ __forceinline__ float group_sum(float s) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// LANES lanes hold one head in pieces of VEC values. blockIdx.y: 0 = q, 1 = k.
// kUnroll heads of a lane group are in flight at once: one load a lane and 2,048
// threads an SM are about the 35 KB that HBM's latency needs, and the table's
// barriers leave gaps, so several are taken.
template <typename T, int VEC, int LANES, bool BWD>
__global__ void __launch_bounds__(kThreads) qk_piece_kernel(Args a) {
  extern __shared__ float2 tab[];
  const int which = blockIdx.y, H = a.heads[which];
  const T *x = static_cast<const T *>(a.x[which]);
  const T *dy = static_cast<const T *>(a.dy[which]);
  T *out = static_cast<T *>(a.out[which]);
  const float *w = a.w[which];
  constexpr int kGroups = kThreads / LANES;
  const int group = threadIdx.x / LANES, gl = threadIdx.x % LANES, i0 = gl * VEC;
  const bool in = i0 < a.N;
  const int half = a.rot / 2;
  float wv[VEC], dw[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    wv[e] = (w && in) ? w[i0 + e] : 1.f;
    dw[e] = 0.f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * a.tile; t0 < a.rows; t0 += (int64_t)gridDim.x * a.tile) {
    const int nt = (int)(a.rows - t0 < a.tile ? a.rows - t0 : a.tile);
    if (half) {
      __syncthreads();
      fill_angles(a, t0, nt, tab);
      __syncthreads();
    }
    const int items = nt * H;
    // every lane of a warp takes part in each shuffle: the loop bound is the block's
    for (int it0 = 0; it0 < items; it0 += kGroups * kUnroll) {
      float v[kUnroll][VEC], d[kUnroll][VEC];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int it = it0 + u * kGroups + group;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[u][e] = d[u][e] = 0.f;
        if (it < items && in) {
          const int64_t at = (t0 * H + it) * a.N + i0;
          load_piece<T, VEC>(x + at, v[u]);
          if (BWD) load_piece<T, VEC>(dy + at, d[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (it0 + u * kGroups >= items) break;
        const int it = it0 + u * kGroups + group;
        const float2 *row = tab + (it < items ? it / H : 0) * half;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s = fmaf(v[u][e], v[u][e], s);
        s = group_sum<LANES>(s);
        const float r = 1.f / sqrtf(fmaf(s, a.share, a.eps));
        if (!BWD) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[u][e] = v[u][e] * r * wv[e];
          if (half) turn_piece<VEC, LANES>(v[u], i0, a, row, 1.f);
          if (it < items && in) store_piece<T, VEC>(out + (t0 * H + it) * a.N + i0, v[u]);
        } else {
          if (half) turn_piece<VEC, LANES>(d[u], i0, a, row, -1.f);
          float dot = 0.f;
          if (it < items) {  // a group behind the last head holds zeros, and r may be infinite there
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              const float xh = v[u][e] * r;
              if (in) dw[e] = fmaf(d[u][e], xh, dw[e]);
              d[u][e] *= wv[e];
              v[u][e] = xh;
              dot = fmaf(d[u][e], xh, dot);
            }
          }
          if (!in) dot = 0.f;
          dot = group_sum<LANES>(dot) * a.share;
#pragma unroll
          for (int e = 0; e < VEC; ++e) d[u][e] = r * (d[u][e] - v[u][e] * dot);
          if (it < items && in) store_piece<T, VEC>(out + (t0 * H + it) * a.N + i0, d[u]);
        }
      }
    }
  }
  if (BWD && a.part[which]) {
    // the block's share of dw: lane groups added in a fixed order
    __shared__ float acc[kThreads / LANES][LANES * VEC + 1];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[group][i0 + e] = dw[e];
    __syncthreads();
    for (int i = threadIdx.x; i < a.N; i += kThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int g = 0; g < kThreads / LANES; ++g) s += acc[g][i];
      a.part[which][(int64_t)blockIdx.x * a.N + i] = s;
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
      fill_angles(a, t0, nt, tab);
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
      const float r = 1.f / sqrtf(fmaf(group_sum<32>(s), a.share, a.eps));
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

// dw[i] = the blocks' shares in a fixed order, in double: 32 slices of the blocks
// side by side, then the slices. One block for q, one for k.
__global__ void __launch_bounds__(1024) qk_weight_kernel(const float *pq, const float *pk, int nblk, int N, float *dwq,
                                                         float *dwk) {
  const float *p = blockIdx.x ? pk : pq;
  float *dw = blockIdx.x ? dwk : dwq;
  if (!p || !dw) return;
  __shared__ double acc[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  for (int i0 = 0; i0 < N; i0 += 32) {
    const int i = i0 + lane;
    double s = 0;
    if (i < N)
      for (int b = slice; b < nblk; b += 32) s += p[(int64_t)b * N + i];
    acc[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && i < N) {
      double t = 0;
      for (int k = 0; k < 32; ++k) t += acc[k][lane];
      dw[i] = (float)t;
    }
    __syncthreads();
  }
}

template <typename T, int VEC, bool BWD>
bool launch_lanes(const Args &a, dim3 grid, size_t smem, cudaStream_t st) {
  const int pieces = a.N / VEC;
  if (pieces <= 4) qk_piece_kernel<T, VEC, 4, BWD><<<grid, kThreads, smem, st>>>(a);
  else if (pieces <= 8) qk_piece_kernel<T, VEC, 8, BWD><<<grid, kThreads, smem, st>>>(a);
  else if (pieces <= 16) qk_piece_kernel<T, VEC, 16, BWD><<<grid, kThreads, smem, st>>>(a);
  else if (pieces <= 32) qk_piece_kernel<T, VEC, 32, BWD><<<grid, kThreads, smem, st>>>(a);
  else return false;
  return true;
}

// Whether heads can be moved in pieces of `vec` values of `size` bytes.
bool pieces_fit(const Args &a, int vec, int size, bool bwd) {
  if (a.N % vec || a.N / vec > 32) return false;
  if (a.rot && !a.interleaved && (a.rot / 2) % vec) return false;
  for (int i = 0; i < 2; ++i) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.x[i]) | reinterpret_cast<uintptr_t>(a.out[i]) |
                          (bwd ? reinterpret_cast<uintptr_t>(a.dy[i]) : 0);
    if (all % (vec * size)) return false;
  }
  return true;
}

template <bool BWD>
cudaError_t launch(const Args &a, int io_t, int blocks, cudaStream_t st) {
  const dim3 grid(blocks, 2);
  const size_t smem = sizeof(float2) * a.tile * (a.rot / 2);
  if (io_t == PDSSM_BF16) {
    using T = __nv_bfloat16;
    if (pieces_fit(a, 8, 2, BWD)) launch_lanes<T, 8, BWD>(a, grid, smem, st);
    else if (pieces_fit(a, 4, 2, BWD)) launch_lanes<T, 4, BWD>(a, grid, smem, st);
    else qk_value_kernel<T, BWD><<<grid, kThreads, smem, st>>>(a);
  } else {
    if (pieces_fit(a, 4, 4, BWD)) launch_lanes<float, 4, BWD>(a, grid, smem, st);
    else qk_value_kernel<float, BWD><<<grid, kThreads, smem, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

// Tokens a tile: up to 8 share one table of angles and one pair of barriers, fewer
// when that would leave SMs without a block.
static int qk_tile(int64_t rows) { return (int)std::min<int64_t>(kMaxTile, std::max<int64_t>(1, rows / (148 * 4))); }

int qk_norm_blocks(int64_t rows) {
  const int64_t tiles = (rows + qk_tile(rows) - 1) / qk_tile(rows);
  return (int)std::min<int64_t>(tiles, 148 * 4);
}

cudaError_t launch_qk_norm(const QkNormArgs &q, bool bwd, cudaStream_t st) {
  Args a{};
  a.rows = q.rows; a.seqlen = q.seqlen;
  a.N = (int)q.N; a.rot = q.rot; a.interleaved = q.interleaved; a.tile = qk_tile(q.rows);
  a.share = q.l2 ? 1.f : 1.f / (float)q.N;
  a.eps = q.eps;
  a.inv_freq = q.inv_freq; a.positions = q.positions;
  const int blocks = qk_norm_blocks(q.rows);
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
    qk_weight_kernel<<<2, 1024, 0, st>>>(a.part[0], a.part[1], blocks, a.N, q.dw[0], q.dw[1]);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = trace_after(st);
  }
  return e;
}

}  // namespace pdssm
