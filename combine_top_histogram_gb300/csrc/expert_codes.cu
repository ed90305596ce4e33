// expert_codes.cu -- what the int8 experts do in memory beside their products.
//
// k_expert_quantise: codes and scales of h, the gated experts' result: for each
// row of the segments s = amax/127 over its F values and codes = RNE(h / s). The
// scale needs the whole row, whose columns many CTAs computed, so h comes
// through memory in fp32 (a rounded h would move codes that lie near a tie). One
// CTA, or of short rows a warp, takes a row at a time, holds it in registers (up to
// 16 values a thread) while its largest magnitude is found, and writes the codes:
// every value of up to 2048 (of a warp's, 512) is read once.
//
// k_widen: codes as fp16, for the products of many rows an expert. It moves three
// bytes a code at HBM's rate; the products that read them then run at the fp16
// rate, while the kernel that converts on its way takes 1010 cycles and more
// where the products alone take 768 (expert_int8.cu). Gated,
// 8 experts and 65536 rows, Zipf(1.2), H = 4096, F = 1408: 1022 us converting on the
// way, 973 with codes widened first, each call on its own (of the launches of the second, under
// the profiler: widening 147 + 51, products 710, quantising 81); back to back 1232 / 1187.
#include <cuda_runtime.h>
#include <stdint.h>

#include "expert_internal.cuh"
#include "expert_math.cuh"
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

// Two quotients v / s rounded to nearest, y = RN(1 / s): two corrections of the
// product by the reciprocal, as minus_quotient in expert_gemm.cu has them, for s
// between 2^-64 and 2^64 (with an IEEE division of each value this kernel takes
// 46 us, with these 20: 10944 rows of 2048).
__device__ __forceinline__ float2 quotient(float2 v, float s, float y) {
  const float2 ns = make_float2(-s, -s), yy = make_float2(y, y);
  float2 q = __fmul2_rn(v, yy);
#pragma unroll
  for (int i = 0; i < 2; ++i) q = __ffma2_rn(__ffma2_rn(ns, q, v), yy, q);
  return q;
}

// |v / s| is at most 127 or so: adding 1.5 * 2^23 rounds it to an integer,
// ties to even, whose low byte is the code. Where s is one of the least numbers there
// are, it may be rounded so far down that the quotient of the row's largest value passes
// 127 (190 times the least, s = once that): codes end at 127.
__device__ __forceinline__ uint32_t codes4(const float4 v, float s, float y) {
  float2 a, b;
  if (y != 0.0f) {
    a = quotient(make_float2(v.x, v.y), s, y);
    b = quotient(make_float2(v.z, v.w), s, y);
  } else {
    const auto q = [&](float x) { return fminf(fmaxf(__fdiv_rn(x, s), -127.0f), 127.0f); };
    a = make_float2(q(v.x), q(v.y));
    b = make_float2(q(v.z), q(v.w));
  }
  const float2 big = make_float2(12582912.0f, 12582912.0f);
  a = __fadd2_rn(a, big);
  b = __fadd2_rn(b, big);
  return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                     __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
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

// The segments' rows: from the first offset to the largest, held to
// [0, rows_max], as the products hold them.
__device__ __forceinline__ void segment_rows(const ExpertArgs& p, uint32_t* buf, int& first,
                                             int& end) {
  const int most = (int)p.rows_max;
  first = min(max(__ldg(p.offset), 0), most);
  end = 0;
  for (int e = threadIdx.x; e <= p.E; e += kThreads) end = max(end, min(__ldg(p.offset + e), most));
  end = (int)cta_max((uint32_t)end, buf);
}

// 16 codes to 32 bytes of fp16. The rows of all segments (per: units of a row),
// or with WEIGHTS the matrix of expert blockIdx.y (per: its units), unless it
// has no rows: where the offset after it is not above its own, none can be in range.
template <bool WEIGHTS>
__global__ void __launch_bounds__(kThreads)
    k_widen(const ExpertArgs p, const uint4* __restrict__ in, uint4* __restrict__ out,
            long long per) {
  __shared__ uint32_t buf[kWarps];
  pdl_wait();
  long long at, end;
  if (WEIGHTS) {
    if (__ldg(p.offset + blockIdx.y + 1) <= __ldg(p.offset + blockIdx.y)) return;
    at = per * blockIdx.y;
    end = at + per;
  } else {
    int first, last;
    segment_rows(p, buf, first, last);
    at = per * first;
    end = per * last;
  }
  constexpr int kAhead = 4;
  for (at += (long long)blockIdx.x * kAhead * kThreads + threadIdx.x; at < end;
       at += (long long)gridDim.x * kAhead * kThreads) {
    uint4 c[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      c[i] = at + i * kThreads < end ? __ldcs(in + at + i * kThreads) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (at + i * kThreads >= end) break;
      const uint2 a = int8_to_f16(c[i].x), b = int8_to_f16(c[i].y), d = int8_to_f16(c[i].z),
                  e = int8_to_f16(c[i].w);
      uint4* o = out + 2 * (at + i * kThreads);
      o[0] = make_uint4(a.x, a.y, b.x, b.y);
      o[1] = make_uint4(d.x, d.y, e.x, e.y);
    }
  }
}

// WARPS of a row: all of the CTA's, or one, which needs no barrier (short rows).
template <int WARPS>
__global__ void __launch_bounds__(kThreads)
    k_expert_quantise(const ExpertArgs p, const float* __restrict__ h, int8_t* __restrict__ codes,
                      float* __restrict__ scale) {
  constexpr int kRow = WARPS * 32, kRows = kThreads / kRow;
  __shared__ uint32_t buf[3][kWarps];
  const int tid = threadIdx.x % kRow, n = p.F >> 2;
  pdl_wait();
  int first, end, par = 0;
  segment_rows(p, buf[2], first, end);
  for (long long r = (long long)first + blockIdx.x * kRows + threadIdx.x / kRow; r < end;
       r += (long long)gridDim.x * kRows, par ^= 1) {
    const float4* row = reinterpret_cast<const float4*>(h + r * p.F);
    float4 v[kHeld];
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = tid + i * kRow;
      v[i] = c < n ? __ldcs(row + c) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) m = max4(m, v[i]);
    for (int c = tid + kHeld * kRow; c < n; c += kRow) m = max4(m, __ldg(row + c));
    m = WARPS == 1 ? __reduce_max_sync(~0u, m) : cta_max(m, buf[par]);
    const bool finite = m < 0x7f800000u;
    const float s = finite ? __fdiv_rn(__uint_as_float(m), 127.0f) : __uint_as_float(m);
    const bool any = finite && s > 0.0f;
    const float y = s >= 0x1p-64f && s <= 0x1p64f ? __frcp_rn(s) : 0.0f;
    uint32_t* out = reinterpret_cast<uint32_t*>(codes + r * p.F);
    if (tid == 0) scale[r] = s;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = tid + i * kRow;
      if (c < n) out[c] = any ? codes4(v[i], s, y) : 0u;
    }
    for (int c = tid + kHeld * kRow; c < n; c += kRow)
      out[c] = any ? codes4(__ldg(row + c), s, y) : 0u;
  }
}

}  // namespace

cudaError_t launch_widen_rows(const ExpertArgs& p, const void* a, uint16_t* x16, int num_sms,
                              cudaStream_t st) {
  return launch_pdl(k_widen<false>, dim3(16u * num_sms), dim3(kThreads), 0, st, p,
                    static_cast<const uint4*>(a), reinterpret_cast<uint4*>(x16),
                    (long long)p.K / 16);
}

cudaError_t launch_widen_weights(const ExpertArgs& p, long long weight_rows, const void* b,
                                 uint16_t* w16, int num_sms, cudaStream_t st) {
  const unsigned each = (16u * num_sms + p.E - 1) / p.E;
  return launch_pdl(k_widen<true>, dim3(each, p.E), dim3(kThreads), 0, st, p,
                    static_cast<const uint4*>(b), reinterpret_cast<uint4*>(w16),
                    weight_rows * (p.K / 16));
}

cudaError_t launch_expert_quantise(const ExpertArgs& p, const float* h, int8_t* codes,
                                   float* scale, int num_sms, cudaStream_t st) {
  const long long most = 16ll * num_sms;
  // one warp / four (us, with the products, means of 60 calls within 0.1; H = 256): E = 11, 3507
  // rows each, F = 464 62.3 / 80.8 (H = 368), E = 8, 4000 rows, F = 640 56.2 / 70.4, F = 896
  // 76.7 / 84.8, 1000 rows, F = 1008 33.4 / 35.1; from some 1200 on both take the same
  // (F = 1264 39.6 / 39.6), and longer rows are read twice by one warp
  if (p.F <= 1024) {
    const long long ctas = (p.rows_max + kWarps - 1) / kWarps;
    return launch_pdl(k_expert_quantise<1>, dim3((unsigned)(ctas < most ? ctas : most)),
                      dim3(kThreads), 0, st, p, h, codes, scale);
  }
  const unsigned ctas = (unsigned)(p.rows_max < most ? p.rows_max : most);
  return launch_pdl(k_expert_quantise<kWarps>, dim3(ctas), dim3(kThreads), 0, st, p, h, codes,
                    scale);
}

}  // namespace moe
