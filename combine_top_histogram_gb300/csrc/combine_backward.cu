// combine_backward.cu -- the gradients of the weighted top-k sum.
//
// out[g] = sum_j w[g,j] y[inv[g,j]], so with dout[g] the gradient of out[g]
//   dy[inv[g,j]] = w[g,j] dout[g]            (each receive row has one slot)
//   dw[g,j]      = <dout[g], y[inv[g,j]]>    (0 for masked and dropped slots)
//
// One pass: a CTA takes a token at a time; each thread loads its 16-byte pieces
// of dout[g] and, for every slot, the same pieces of the slot's y row (a few
// pieces of all slots before the first product), adds their products in fp32
// and writes the scaled pieces to the slot's dy row. The slots of the CTA's
// next token are loaded beside this one's rows. The k sums are then reduced
// over the CTA in a fixed order (no atomics: the same inputs give the same
// bits). Bound by HBM: y in, dy out, dout once (32768 tokens, top-2, H = 4096:
// 191 us, 6.75 TB/s, the rate of a copy; with one piece of a row at a time and
// the slots loaded in the token's turn 227; 1024 tokens, top-8, H = 7168: 42 us,
// 5.9 TB/s, one wave of CTAs and the launch).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

__device__ __forceinline__ uint32_t scale2(uint32_t u, float w) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(__fmul_rn(w, lo_f(u)), __fmul_rn(w, hi_f(u)));
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float dot8(const uint4 a, const uint4 b, float acc) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    acc = __fmaf_rn(lo_f(x[q]), lo_f(y[q]), acc);
    acc = __fmaf_rn(hi_f(x[q]), hi_f(y[q]), acc);
  }
  return acc;
}

// K slots at a time: K == k for the common k, 8 otherwise (any k). V pieces of
// a row at a time, by kThreads threads.
template <int K, int V, int kThreads>
__global__ void __launch_bounds__(kThreads) k_combine_backward(const CombineBackwardArgs p) {
  __shared__ int rows_buf[2][MOE_MAX_TOPK];
  __shared__ float w_buf[2][MOE_MAX_TOPK];
  __shared__ float part[2][kThreads / 32][MOE_MAX_TOPK];
  const int nvec = p.H >> 3, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int par = 0, row_next = -1;
  float w_next = 0.0f;
  const auto fetch = [&](long long g) {
    if (tid < p.k && g < p.T) {
      row_next = __ldg(p.inv + g * p.k + tid);
      w_next = __ldg(p.w + g * p.k + tid);
    }
  };
  pdl_wait();
  fetch(blockIdx.x);
  for (long long g = blockIdx.x; g < p.T; g += gridDim.x) {
    int* rows_s = rows_buf[par];
    float* w_s = w_buf[par];
    if (tid < p.k) {
      // A row past the buffers (tokens that a chunked dispatch has left out keep the
      // rows of an earlier layout) is reported and taken as no slot, in every build.
      if (row_next >= p.rows) {
        atomicOr(p.status, MOE_STATUS_BOUNDS);
        row_next = -1;
      }
      rows_s[tid] = row_next >= 0 ? row_next : -1;
      w_s[tid] = w_next;
    }
    __syncthreads();
    fetch(g + gridDim.x);
    const uint4* d = reinterpret_cast<const uint4*>(p.dout + g * p.H);
    for (int j0 = 0; j0 < p.k; j0 += K) {
      float acc[K];
#pragma unroll
      for (int j = 0; j < K; ++j) acc[j] = 0.0f;
      for (int v0 = tid; v0 < nvec; v0 += V * kThreads) {
        uint4 dv[V], yv[V][K];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int v = v0 + i * kThreads;
          if (v >= nvec) break;
          dv[i] = __ldg(d + v);
#pragma unroll
          for (int j = 0; j < K; ++j) {
            const int r = j0 + j < p.k ? rows_s[j0 + j] : -1;
            yv[i][j] = r >= 0 ? __ldcs(reinterpret_cast<const uint4*>(p.y + (long long)r * p.H) + v)
                              : make_uint4(0u, 0u, 0u, 0u);
          }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int v = v0 + i * kThreads;
          if (v >= nvec) break;
#pragma unroll
          for (int j = 0; j < K; ++j) {
            const int r = j0 + j < p.k ? rows_s[j0 + j] : -1;
            if (r < 0) continue;
            acc[j] = dot8(dv[i], yv[i][j], acc[j]);
            const float w = w_s[j0 + j];
            __stcs(reinterpret_cast<uint4*>(p.dy + (long long)r * p.H) + v,
                   make_uint4(scale2(dv[i].x, w), scale2(dv[i].y, w), scale2(dv[i].z, w),
                              scale2(dv[i].w, w)));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < K; ++j) {
        for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(~0u, acc[j], o);
        if (lane == 0 && j0 + j < p.k) part[par][warp][j0 + j] = acc[j];
      }
    }
    __syncthreads();
    if (tid < p.k) {
      float sum = 0.0f;
      if (rows_s[tid] >= 0) {
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) sum += part[par][w][tid];
      }
      p.dw[g * p.k + tid] = sum;
    }
    par ^= 1;  // the other buffers next: these are read until the next token's barriers
  }
}

template <int K, int V>
cudaError_t launch(const CombineBackwardArgs& a, int num_sms, cudaStream_t st) {
  // Few tokens: a CTA's threads share a row more finely, so that its loads take
  // fewer turns (300 tokens, top-8, H = 7168: 15.2 us a pass with 128 threads,
  // under the 10.6 us of the calling program with 512).
  if (a.T <= 2ll * num_sms && a.H > 1024)
    return launch_pdl(k_combine_backward<K, 1, 512>, dim3((unsigned)a.T), dim3(512), 0, st, a);
  const long long cap = (long long)num_sms * 16;
  const dim3 grid((unsigned)(a.T < cap ? a.T : cap));
  return launch_pdl(k_combine_backward<K, V, 128>, grid, dim3(128), 0, st, a);
}

}  // namespace

cudaError_t launch_combine_backward(const CombineBackwardArgs& a, int num_sms, cudaStream_t st) {
  switch (a.k) {
    case 1: return launch<1, 4>(a, num_sms, st);
    case 2: return launch<2, 4>(a, num_sms, st);
    case 4: return launch<4, 2>(a, num_sms, st);
    default: return launch<8, 1>(a, num_sms, st);
  }
}

}  // namespace moe
