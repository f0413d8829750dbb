// round16.cuh — fp32 to the cache's 16-bit types, for the kernels behind
// moe_batch.h.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

// Two values rounded to fp16 (kF16) or bf16, to nearest even, lo in the lower half.
template <bool kF16>
MOE_DEV uint32_t round16(float lo, float hi) {
  if constexpr (kF16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    return pack_bf16x2(lo, hi);
  }
}

}  // namespace moe
