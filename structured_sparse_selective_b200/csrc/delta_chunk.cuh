// What the chunked kernels of the gated delta rule share: the record's layout, splits
// into bf16 parts and bounded waits.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace pdssm {

constexpr int kChunk = 64;
// A 64 x 64 bf16 operand, element (row c, column j): (j / 8) * 1024 + c * 16 + (j % 8) * 2.
// Read K-major it is [rows c][k = j], read MN-major [k = c][columns j].
constexpr int kSquare = kChunk * kChunk * 2;
constexpr int kChunkGroup = kChunk * 16 + 16;  // bytes of eight columns of K or Q; 16 more spread the banks
// exp(G), exp(G_64 - G), beta, exp(G_64) in two parts (in turn), and G to the base 2 as two floats, 64 values each
constexpr int kScalars = 6 * kChunk * 4;
// Record of a chunk: Te (3 parts), backward also Tb (3 parts), A (2 parts, backward 3), scalars.
constexpr int delta_a_parts(bool bwd) { return bwd ? 3 : 2; }
constexpr int64_t delta_record_bytes(bool bwd) { return ((bwd ? 6 : 3) + delta_a_parts(bwd)) * (int64_t)kSquare + kScalars; }

// bf16 parts of two values, packed (x in the lower half): x = hi + mid + lo up to 2^-24 of x.
// Rounding to bf16 and the differences are exact, so each part has the next 8 bits.
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ float low_half(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float high_half(uint32_t p) { return __uint_as_float(p & 0xffff0000u); }
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16(x, y);
  lo = pack_bf16(x - low_half(hi), y - high_half(hi));
}
__device__ __forceinline__ void split3(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  hi = pack_bf16(x, y);
  x -= low_half(hi);
  y -= high_half(hi);
  mid = pack_bf16(x, y);
  lo = pack_bf16(x - low_half(mid), y - high_half(mid));
}

// The first min(n, 8) values at p, any alignment, zeros behind them.
__device__ __forceinline__ uint4 gather8(const __nv_bfloat16 *p, int n) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = 2 * i < n ? *reinterpret_cast<const uint16_t *>(p + 2 * i) : 0;
    const uint32_t y = 2 * i + 1 < n ? *reinterpret_cast<const uint16_t *>(p + 2 * i + 1) : 0;
    w[i] = x | (y << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The rows [row0, row0 + 64) of head `head` of x [rows][heads][n] as an operand in shared
// memory, element (step c, column j): (j / 8) * GROUP + c * ROW + (j % 8) * 2, by THREADS
// threads. `wide`: 16-byte asynchronous copies (n a multiple of 8, x aligned to 16 bytes).
// Zeros behind the `live` rows and the n columns. A thread has one group of columns and
// every THREADS / NG-th row: two additions a copy (with the place worked out for each copy
// a chunk's copies took 4,000 to 8,000 cycles to ask for, longer than the chunk).
template <int NG, int GROUP, int ROW, int THREADS>
__device__ __forceinline__ void load_tile(uint8_t *dst, const __nv_bfloat16 *x, int64_t row0, int64_t heads, int64_t head, int64_t n,
                                          int64_t n0, int live, bool wide, int tid) {
  constexpr int kStep = THREADS / NG;
  static_assert(THREADS % NG == 0 && kChunk % kStep == 0, "whole rows");
  const int g = tid % NG, c0 = tid / NG, have = (int)min((int64_t)8 * NG, n - n0);
  const int64_t row = heads * n, step = kStep * row;
  const __nv_bfloat16 *src = x + (row0 * heads + head) * n + n0 + 8 * g + c0 * row;
  uint8_t *to = dst + g * GROUP + c0 * ROW;
  if (wide && live == kChunk && 8 * g < have) {
#pragma unroll
    for (int c = 0; c < kChunk / kStep; ++c, src += step) sm100::cp_async16(to + c * kStep * ROW, src);
  } else {
    for (int c = c0; c < kChunk; c += kStep, src += step, to += kStep * ROW) {
      if (wide && c < live && 8 * g < have) sm100::cp_async16(to, src);
      else *reinterpret_cast<uint4 *>(to) = c < live && 8 * g < have ? gather8(src, have - 8 * g) : make_uint4(0, 0, 0, 0);
    }
  }
}

// 2^x, off by at most about 2^-22 of it.
__device__ __forceinline__ float decay2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

constexpr uint64_t kShortNs = 1000000, kOwnNs = 2000000000ull;

// Waits for the barrier's phase for at most limit_ns; then records the timeout and returns false.
// A wait on another role (OWN false) also ends when the call has run out of time anywhere.
template <bool OWN>
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, uint32_t *err, uint64_t limit_ns) {
  const uint64_t t0 = now_ns();
  // the waiting instruction may sleep longer than a short limit
  while (!(limit_ns < kShortNs ? sm100::mbar_test_wait(bar, parity) : sm100::mbar_try_wait_sleep(bar, parity, 2000))) {
    if (now_ns() - t0 >= limit_ns || (!OWN && (*reinterpret_cast<volatile uint32_t *>(err) & kErrTimeout))) {
      flag_error(err, kErrTimeout);
      return false;
    }
  }
  return true;
}
// On another role.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, uint32_t *err, uint64_t limit_ns) {
  return sm100::mbar_try_wait(bar, parity) || wait_slow<false>(bar, parity, err, limit_ns);
}
// On the caller's own copies or products in flight. The tries in place rarely leave the call to be
// made (the gradients' launch of 256 sequences of 2,048 steps, 64 x 64: 371 -> 330 us; in the chains
// of the roles' waits the loop is slower, 150 -> 177 us).
__device__ __forceinline__ bool wait_own(uint64_t *bar, uint32_t parity, uint32_t *err) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (sm100::mbar_try_wait(bar, parity)) return true;
  return wait_slow<true>(bar, parity, err, kOwnNs);
}

// True in all THREADS of some whole warps (by a barrier of their own) if ok is true in all.
template <int THREADS>
__device__ __forceinline__ bool all_of(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)ok), "n"(THREADS)
      : "memory");
  return r != 0;
}

// W fp32 values as packed bf16 parts 0 .. PARTS - 1 into columns col, col + stride, ... of the
// thread's row (col already at the thread's or the warp's part), 16 values at a time: the parts
// of 64 at once would take 96 registers.
template <int PM, int W, int PARTS>
__device__ __forceinline__ void store_parts(uint32_t taddr, int stride, const float (&v)[W]) {
#pragma unroll
  for (int j = 0; j < W; j += 16) {
    uint32_t p[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (PARTS == 3) split3(v[j + 2 * i], v[j + 2 * i + 1], p[0][i], p[1][i], p[2][i]);
      else split2(v[j + 2 * i], v[j + 2 * i + 1], p[0][i], p[1][i]);
    }
#pragma unroll
    for (int q = 0; q < PARTS; ++q) sm100::TmemIo<PM, 8, W / 2>::st(taddr + q * stride + j / 2, p[q]);
  }
}

template <int PM, int W>
__device__ __forceinline__ void load_cols(uint32_t taddr, float (&v)[W]) {
  uint32_t r[W];
  sm100::TmemIo<PM, W>::ld(taddr, r);
  sm100::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = __uint_as_float(r[i]);
}

template <int W>
__device__ __forceinline__ void load_scalars(float (&v)[W], const float *p) {
#pragma unroll
  for (int c = 0; c < W; c += 4) {
    const float4 x = *reinterpret_cast<const float4 *>(p + c);
    v[c] = x.x; v[c + 1] = x.y; v[c + 2] = x.z; v[c + 3] = x.w;
  }
}

// x[0 .. n) to rows of `ld` floats at `to`, a column each lane. Rows of PM floats and all W of
// them: the addresses are constants apart.
template <int PM, int W>
__device__ __forceinline__ void store_rows(float *to, int64_t ld, int n, const float (&x)[W]) {
  if (n >= W && ld == PM) {
#pragma unroll
    for (int c = 0; c < W; ++c) to[c * PM] = x[c];
  } else if (n > 0) {
#pragma unroll
    for (int c = 0; c < W; ++c)
      if (c < n) to[c * ld] = x[c];
  }
}

}  // namespace pdssm
