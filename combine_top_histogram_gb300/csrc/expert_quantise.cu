// expert_quantise.cu -- int8 codes and scales of h, the gated experts' result:
// for each row of the segments s = amax/127 over its F values and
// codes = RNE(h / s).
//
// The scale needs the whole row, whose columns many CTAs computed, so h comes
// through memory in fp32 (a rounded h would move codes that lie near a tie). One
// CTA takes a row at a time, holds it in registers (up to 16 values a thread)
// while its largest magnitude is found, and writes the codes: every value is
// read once.
#include <cuda_runtime.h>
#include <stdint.h>

#include "expert_internal.cuh"
#include "internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 4;  // four values each, of a thread

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Largest magnitude, by its bits: infinity is above every number, NaN above that.
__device__ __forceinline__ uint32_t max4(uint32_t m, const float4 v) {
  return max(max(m, max(abs_bits(v.x), abs_bits(v.y))), max(abs_bits(v.z), abs_bits(v.w)));
}

// |v / s| is at most 127 or so: adding 1.5 * 2^23 rounds it to an integer,
// ties to even, whose low byte is the code.
__device__ __forceinline__ uint32_t code_bits(float v, float s) {
  return __float_as_uint(__fadd_rn(__fdiv_rn(v, s), 12582912.0f));
}
__device__ __forceinline__ uint32_t codes4(const float4 v, float s) {
  return __byte_perm(__byte_perm(code_bits(v.x, s), code_bits(v.y, s), 0x0040),
                     __byte_perm(code_bits(v.z, s), code_bits(v.w, s), 0x0040), 0x5410);
}

// The maximum over the CTA; `buf` is not written again before the next barrier but one.
__device__ __forceinline__ uint32_t cta_max(uint32_t m, uint32_t* buf) {
  m = __reduce_max_sync(~0u, m);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) m = max(m, buf[i]);
  return m;
}

__global__ void __launch_bounds__(kThreads)
    k_expert_quantise(const ExpertArgs p, const float* __restrict__ h, int8_t* __restrict__ codes,
                      float* __restrict__ scale) {
  __shared__ uint32_t buf[3][kWarps];
  const int tid = threadIdx.x, n = p.F >> 2;
  pdl_wait();
  // the segments' rows are those from the first offset to the largest, held to
  // [0, rows_max], as the products hold them
  const int most = (int)p.rows_max;
  const int first = min(max(__ldg(p.offset), 0), most);
  int end = 0;
  for (int e = tid; e <= p.E; e += kThreads) end = max(end, min(__ldg(p.offset + e), most));
  end = (int)cta_max((uint32_t)end, buf[2]);
  int par = 0;
  for (long long r = (long long)first + blockIdx.x; r < end; r += gridDim.x, par ^= 1) {
    const float4* row = reinterpret_cast<const float4*>(h + r * p.F);
    float4 v[kHeld];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = tid + i * kThreads;
      v[i] = c < n ? __ldcs(row + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) m = max4(m, v[i]);
    for (int c = tid + kHeld * kThreads; c < n; c += kThreads) m = max4(m, __ldg(row + c));
    m = cta_max(m, buf[par]);
    const bool finite = m < 0x7f800000u;
    const float s = finite ? __fdiv_rn(__uint_as_float(m), 127.0f) : __uint_as_float(m);
    const bool any = finite && s > 0.0f;
    uint32_t* out = reinterpret_cast<uint32_t*>(codes + r * p.F);
    if (tid == 0) scale[r] = s;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = tid + i * kThreads;
      if (c < n) out[c] = any ? codes4(v[i], s) : 0u;
    }
    for (int c = tid + kHeld * kThreads; c < n; c += kThreads)
      out[c] = any ? codes4(__ldg(row + c), s) : 0u;
  }
}

}  // namespace

cudaError_t launch_expert_quantise(const ExpertArgs& p, const float* h, int8_t* codes,
                                   float* scale, int num_sms, cudaStream_t st) {
  const long long most = 16ll * num_sms;
  const int grid = (int)(p.rows_max < most ? p.rows_max : most);
  return launch_pdl(k_expert_quantise, dim3(grid), dim3(kThreads), 0, st, p, h, codes, scale);
}

}  // namespace moe
