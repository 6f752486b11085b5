// What the gated delta rule's kernels share.
//
// Per (sequence b, value head h), with key head h / (heads / qk_heads), a_t = exp(g_t):
//   e_t = v_t - a_t H_{t-1}^T k_t           (what the faded memory lacks of the value)
//   H_t = a_t H_{t-1} + beta_t k_t e_t^T    (N x P)
//   y_t = scale H_t^T q_t
// and backwards, with X_t = dLoss/dH_t before the step is undone:
//   X_t = X'_t + scale q_t dy_t^T,  du_t = X_t^T k_t,  dv_t = beta_t du_t,
//   X'_{t-1} = a_t (X_t - k_t dv_t^T)
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pdssm {

// A decay below exp(-110) is 0 in fp32; the clamp keeps sums of log decays finite,
// so that -inf (the state is dropped) is an ordinary value. NaN stays NaN.
__device__ __forceinline__ float clamp_gate(float g) { return g < -110.f ? -110.f : g; }

// exp(g) as a float and what it lacks: exp(g) = d.a + d.rest, |d.rest| <= 2^-25 (2^-24 above 1). A state of slow decay
// is multiplied by the same factors thousands of times, so half a step of the float, 2^-25, each time becomes 2^-11 of
// the state after 2^14 steps. Near 1 the rest is known from exp(g) - 1, by its series (off by less than 2^-33 of 1);
// what decays by more than exp(-1/8) is forgotten in a few steps. UNIFORM: all lanes have the same g and go one way
// (one token of 64 sequences x 32 heads, 128 x 64: 30.5 -> 27.5 us; where lanes have steps of their own the branch makes
// the chains of steps slower, 338 -> 379 us for 32 sequences of 4,000 steps, 32 x 32).
struct Decay {
  float a, rest;
};
template <bool UNIFORM>
__device__ __forceinline__ Decay decay_of(float g) {
  g = clamp_gate(g);
  const bool near = fabsf(g) < 0.125f;
  if (UNIFORM && !near) return {expf(g), 0.f};
  float m = fmaf(g, 1.f / 6, 1.f);
  m = fmaf(g * (1.f / 5), m, 1.f);
  m = fmaf(g * (1.f / 4), m, 1.f);
  m = fmaf(g * (1.f / 3), m, 1.f);
  m = fmaf(g * (1.f / 2), m, 1.f) * g;
  const float a = 1.f + m;  // a - 1 and what m has more are exact, |m| < 1
  if (UNIFORM) return {a, m - (a - 1.f)};
  return {near ? a : expf(g), near ? m - (a - 1.f) : 0.f};
}

// Steps of sequence b that count: its length clamped to [0, L], or L.
__device__ __forceinline__ int64_t live_steps(const int32_t *lengths, int64_t b, int64_t L) {
  if (!lengths) return L;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : (n > L ? L : n);
}

__device__ __forceinline__ float load_any(const void *p, int64_t i, bool bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_any(void *p, int64_t i, bool bf16, float v) {
  if (bf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float *>(p)[i] = v;
}

// Whether a wait of the call has run out so far, anywhere in it.
__device__ __forceinline__ bool timed_out(const uint32_t *err) { return *static_cast<const volatile uint32_t *>(err) & kErrTimeout; }

// NaN over `rows` rows of `cols` values, `ld` apart, from value `at` of p on (nothing where p is null), by `threads`
// threads: what a call whose waits ran out gives back instead of values that are not finished.
static __device__ __noinline__ void fill_nan(void *p, bool bf16, int64_t at, int64_t rows, int64_t ld, int cols, int tid, int threads) {
  if (!p || cols <= 0) return;
  for (int64_t i = tid; i < rows * cols; i += threads) store_any(p, at + i / cols * ld + i % cols, bf16, __int_as_float(0x7fffffff));
}

// Two fp32 values in one register pair; one instruction works on both.
using pair2 = unsigned long long;
__device__ __forceinline__ pair2 pack2(float a, float b) {
  pair2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(pair2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ pair2 fma2(pair2 a, pair2 b, pair2 c) {
  pair2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ pair2 mul2(pair2 a, pair2 b) {
  pair2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace pdssm
