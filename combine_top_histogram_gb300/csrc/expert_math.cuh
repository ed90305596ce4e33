// expert_math.cuh -- the SiLU of the gated feed-forward block. Device code only.
#pragma once

#include <cuda_runtime.h>

namespace moe {

// 1 / (1 + exp(-g)) as 1 / (1 + 2^(-g log2 e)) with the hardware's approximate
// 2^x and reciprocal, each within 2^-22 of the value; the rounded argument adds
// up to |g| 2^-24. A result below 2^-126 (g below -87.3) is flushed to 0, and
// silu(g), there below 2^-119 in magnitude, with it.
__device__ __forceinline__ float sigmoid(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

__device__ __forceinline__ float silu(float g) { return g * sigmoid(g); }

}  // namespace moe
