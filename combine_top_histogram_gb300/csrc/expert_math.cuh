// expert_math.cuh -- the SiLU of the gated feed-forward block. Device code only.
#pragma once

#include <cuda_runtime.h>

namespace moe {

// 1 / (1 + exp(-g)); exp(-g) = +inf gives 0.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// g / (1 + exp(-g)). __fdividef returns 0 for divisors above 2^126 (there the
// quotient is below every value that a product with it could show).
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

}  // namespace moe
