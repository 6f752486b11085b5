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
constexpr int kScalars = 4 * kChunk * 4;  // exp(G), exp(G_64 - G), beta, exp(G_64), 64 floats each
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

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Waits for the barrier's phase for at most limit_ns; then records the timeout and
// returns false (the caller goes on without waiting, on data inside its buffers).
static __device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, uint32_t *err, uint64_t limit_ns) {
  const uint64_t t0 = now_ns();
  while (!sm100::mbar_try_wait_sleep(bar, parity, 2000)) {
    if (now_ns() - t0 > limit_ns) {
      flag_error(err, kErrTimeout);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, uint32_t *err, uint64_t limit_ns) {
  return sm100::mbar_try_wait(bar, parity) || wait_slow(bar, parity, err, limit_ns);
}

}  // namespace pdssm
