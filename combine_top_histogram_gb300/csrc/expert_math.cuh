// expert_math.cuh -- the SiLU of the gated feed-forward block, and int8 codes as
// tensor-core operands. Device code only.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

// Four int8 codes as fp16, exactly, by the well-known way of putting an integer into the low bits
// of a constant's significand and subtracting the constant: with the sign bit turned over a byte is
// code + 128, as the low byte of an fp16 of 1024 it makes 1152 + code, and one
// subtraction leaves the code. In order, .x the first two.
__device__ __forceinline__ uint2 int8_to_f16(uint32_t codes) {
  const uint32_t u = codes ^ 0x80808080u, k = 0x64806480u;  // k: 1152, twice
  uint2 r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r.x) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(k));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r.y) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(k));
  return r;
}

}  // namespace moe
