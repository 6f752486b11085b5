// Argument checks shared by the C-ABI files.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pdssm.h"

namespace pdssm {

inline size_t dtype_size(int dt) {
  switch (dt) {
    case PDSSM_F32: return 4;
    case PDSSM_BF16: return 2;
    case PDSSM_C64: return 8;
    default: return 0;
  }
}

inline bool mul_ok(int64_t a, int64_t b, int64_t *out) { return !__builtin_mul_overflow(a, b, out); }

inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

inline bool aligned(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

inline pdssm_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PDSSM_OK : PDSSM_ERR_CUDA; }

}  // namespace pdssm
