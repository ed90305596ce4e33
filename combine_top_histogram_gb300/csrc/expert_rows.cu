// expert_rows.cu -- the experts' forward products for a few rows (single
// tokens): the same results as expert_gemm.cu's kGated and kDown, organised to
// stream the weights of the experts that have rows as fast as HBM gives them.
//
// With a row or two per expert the work is the weights' bytes. A warp takes two
// groups of 16 weight rows of one expert (16 gate and the same 16 up channels,
// or 32 output channels); S warps of a CTA share one such pair of groups and
// split the reduction axis in pieces of 128 bytes, and the CTA's 8 / S pairs
// are neighbours. S is 8 where there are few groups, so that even one token of
// a small layer spreads over many SMs, and less where there are many, so that
// the start and the end of a CTA are paid for by more bytes (down, e4m3, one
// token of E = 256, top-8, H = 7168, F = 2048: 24.3 us at S = 4, 28.5 at 8).
// A warp's products are mma.sync m16n8 with the weight rows as the 16 and up
// to eight rows of the segment as the 8: the tensor cores take the bytes as
// they are loaded (16 per lane, along K; both operands permute k in the same
// way, which a sum does not see), without conversions and without shared
// memory. More than eight rows are taken in passes that find the weights in
// L2. The S partial sums meet in shared memory in a fixed order.
// e4m3: each 128-channel block is one piece; its products are multiplied by
// the row's and the weight block's fp32 scales before they are added. The 128
// channels that share a scale of h are the S CTAs of one cluster, which
// exchange their rows' largest magnitudes through distributed shared memory.
// int8: codes become fp16 in registers (exact, and so are their products), 5
// instructions for four; whole sums, then the row's and the channel's scale. h
// leaves in fp32, for its scale is the whole row's (expert_codes.cu).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "expert_internal.cuh"
#include "expert_math.cuh"
#include "expert_ptx.cuh"
#include "internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 2;  // pieces loaded before the first product

template <int TYPE>
__device__ __forceinline__ void mma16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (TYPE == kE4m3)
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else if constexpr (TYPE == kInt8)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The products of 16 bytes of each of a lane's weight rows g and g + 8 with as
// many of its receive row. int8 codes become fp16, four k of a word to one
// product of 16 k.
template <int TYPE>
__device__ __forceinline__ void mma_piece(float (&c)[4], const uint4& a, const uint4& b,
                                          const uint4& x) {
  if constexpr (TYPE == kInt8) {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w},
                   xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 fa = int8_to_f16(aw[i]), fb = int8_to_f16(bw[i]), fx = int8_to_f16(xw[i]);
      mma16x8<TYPE>(c, fa.x, fb.x, fa.y, fb.y, fx.x, fx.y);
    }
  } else {
    mma16x8<TYPE>(c, a.x, b.x, a.y, b.y, x.x, x.y);
    mma16x8<TYPE>(c, a.z, b.z, a.w, b.w, x.z, x.w);
  }
}

__device__ __forceinline__ uint4 load_if(const uint8_t* p, bool ok) {
  return ok ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}
// Weights are read once per pass.
__device__ __forceinline__ uint4 stream_if(const uint8_t* p, bool ok) {
  return ok ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}

// The a-th expert that has rows, its first row and its rows; n = 0 if there
// are not so many. Whole CTA. Segments are those of the tile kernels: offsets
// held to [0, rows_max], ends to ascending order. Where some end descends (the
// caller's own offsets; a layout's never do) one thread walks them again.
struct Segment {
  int e, row0, n;
};
__device__ __forceinline__ Segment find_segment(const ExpertArgs& p, int a) {
  __shared__ int warp_count[kWarps];
  __shared__ Segment found;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kPer = MOE_MAX_EXPERTS / kThreads;
  const int per = (p.E + kThreads - 1) / kThreads;  // <= kPer
  const auto offset = [&](int e) { return min(max(__ldg(p.offset + e), 0), (int)p.rows_max); };
  int lo[kPer], n[kPer], count = 0;
  bool descends = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * per + i;
    lo[i] = n[i] = 0;
    if (i < per && e < p.E) {
      lo[i] = offset(e);
      n[i] = offset(e + 1) - lo[i];
    }
    descends |= n[i] < 0;
    count += n[i] > 0;
  }
  int sum = count;
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(~0u, sum, d);
    if (lane >= d) sum += v;
  }
  if (lane == 31) warp_count[warp] = sum;
  if (tid == 0) found = Segment{0, 0, 0};
  if (__syncthreads_or(descends)) {
    if (tid == 0) {
      int top = offset(0), before = 0;
      for (int e = 0; e < p.E; ++e) {
        const int end = max(offset(e + 1), top);
        if (end > top && before++ == a) found = Segment{e, top, end - top};
        top = end;
      }
    }
  } else {
    int before = sum - count;
    for (int w = 0; w < warp; ++w) before += warp_count[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (n[i] > 0) {
        if (before == a) found = Segment{tid * per + i, lo[i], n[i]};
        ++before;
      }
    }
  }
  __syncthreads();
  return found;
}

template <int OP, int TYPE, int S>
__global__ void __launch_bounds__(kThreads, 2)
    k_expert_rows(const ExpertArgs p, const void* a_rows, const void* weights) {
  constexpr bool FP8 = TYPE == kE4m3, INT8 = TYPE == kInt8;
  constexpr bool kQuant = OP == kGated && FP8;
  constexpr int kGroups = kWarps / S;                       // pairs of groups of this CTA
  constexpr int kChannels = kGroups * (OP == kGated ? 16 : 32);
  __shared__ float part[kWarps][2][8 * 16];                 // [row][channel] each
  __shared__ int amax[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  const int per_expert = (p.N + kChannels - 1) / kChannels;
  const Segment seg = find_segment(p, blockIdx.x / per_expert);
  if (seg.n == 0) return;
  const int cta0 = (blockIdx.x % per_expert) * kChannels;  // the CTA's first channel
  const int c0 = cta0 + warp / S * (OP == kGated ? 16 : 32), ks = warp % S;
  // weight rows of this lane: g and g + 8 of each group of 16
  const long long kbytes = (long long)p.K * (TYPE == kBf16 ? 2 : 1);
  const int b_rows = OP == kGated ? 2 * p.F : p.N;
  const uint8_t* wp[4];
  bool w_ok[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = c0 + g + (i & 1) * 8 + (OP == kDown ? (i >> 1) * 16 : 0);
    w_ok[i] = c < p.N;
    const int r = (w_ok[i] ? c : 0) + (OP == kGated && i >= 2 ? p.F : 0);
    wp[i] = static_cast<const uint8_t*>(weights) + ((long long)seg.e * b_rows + r) * kbytes;
  }
  const int pieces = (int)((kbytes + 127) >> 7);
  const float *sb0 = nullptr, *sb1 = nullptr;
  if constexpr (FP8) {
    const int blocks = b_rows >> 7, blk = min(c0, p.N - 1) >> 7;
    sb0 = p.sb + ((long long)seg.e * blocks + blk) * pieces;
    sb1 = OP == kGated ? sb0 + (long long)(p.F >> 7) * pieces : sb0;
  }
  for (int r0 = 0; r0 < seg.n; r0 += 8) {
    const int rows = min(seg.n - r0, 8);
    const long long row0 = (long long)seg.row0 + r0;
    const uint8_t* xp =
        static_cast<const uint8_t*>(a_rows) + (row0 + (g < rows ? g : 0)) * kbytes;
    const float* sa0 = p.sa + (row0 + min(2 * t, rows - 1)) * pieces;
    const float* sa1 = p.sa + (row0 + min(2 * t + 1, rows - 1)) * pieces;
    float acc[2][4] = {};
    uint4 w[kAhead][4][2], x[kAhead][2];
    float s[kAhead][4];
    const auto load = [&](int u, int cu) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const long long at = (long long)cu * 128 + h * 64 + t * 16;
        const bool in = at < kbytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[u][i][h] = stream_if(wp[i] + at, in && w_ok[i]);
        x[u][h] = load_if(xp + at, in && g < rows);
      }
      if constexpr (FP8) {
        const int k = min(cu, pieces - 1);
        const float a0 = __ldg(sa0 + k), a1 = __ldg(sa1 + k);
        const float b0 = __ldg(sb0 + k), b1 = __ldg(sb1 + k);
        s[u][0] = a0 * b0;
        s[u][1] = a1 * b0;
        s[u][2] = a0 * b1;
        s[u][3] = a1 * b1;
      }
    };
    const auto multiply = [&](int u) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v[4] = {};
        float(&d)[4] = FP8 ? v : acc[j];
#pragma unroll
        for (int h = 0; h < 2; ++h) mma_piece<TYPE>(d, w[u][2 * j][h], w[u][2 * j + 1][h], x[u][h]);
        if constexpr (FP8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(v[i], s[u][2 * j + (i & 1)], acc[j][i]);
        }
      }
    };
    if constexpr (INT8) {
      // The conversions keep a warp busy for long, so the next piece is loaded into
      // a place as soon as that is free (us of one token, E = 256, top-8, H = 7168, F = 2048, the
      // caches empty, without / with: gated 84.5 / 48.0, down 56.1 / 28.5; the other types
      // lose by it, e4m3 49.0 / 55.5 and 28.6 / 29.3).
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load(u, ks + u * S);
      for (int c = ks; c < pieces; c += S * kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (c + u * S < pieces) multiply(u);
          load(u, c + (u + kAhead) * S);
        }
      }
    } else {
      for (int c = ks; c < pieces; c += S * kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) load(u, c + u * S);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          if (c + u * S >= pieces) break;
          multiply(u);
        }
      }
    }
    // lane holds rows 2t and 2t + 1 of channels g and g + 8
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        part[warp][j][(2 * t + (i & 1)) * 16 + g + (i >> 1) * 8] = acc[j][i];
    if (kQuant && tid < 8) amax[tid] = 0;
    __syncthreads();
    // this thread's results: [row][channel], kPer of them
    constexpr int kPer = 8 * kChannels / kThreads > 0 ? 8 * kChannels / kThreads : 1;
    float out[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = tid + i * kThreads, r = at / kChannels, ch = at % kChannels;
      if (8 * kChannels < kThreads && r >= 8) break;
      const int group = ch / (OP == kGated ? 16 : 32) * S, j = OP == kDown ? (ch >> 4) & 1 : 0;
      const int k = r * 16 + (ch & 15);
      float v = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int w = 0; w < S; ++w) {
        v += part[group + w][j][k];
        if (OP == kGated) v1 += part[group + w][1][k];
      }
      const bool mine = r < rows && cta0 + ch < p.N;
      const long long o = (row0 + r) * p.N + cta0 + ch;
      if constexpr (INT8) {  // whole sums of codes, then the row's and the channel's scales
        if (mine) {
          const float sr = __ldg(p.sa + row0 + r);
          const float* sc = p.sb + (long long)seg.e * b_rows + cta0 + ch;
          v = v * sr * __ldg(sc);
          if (OP == kGated) v1 = v1 * sr * __ldg(sc + p.F);
        }
      }
      if constexpr (OP == kDown) {
        if (mine) static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v);
      } else {
        out[i] = silu(v) * v1;
        if constexpr (kQuant) {  // the largest magnitude, by its bits: NaN is above all
          if (mine) atomicMax(&amax[r], __float_as_int(fabsf(out[i])));
        } else if constexpr (INT8) {
          if (mine) static_cast<float*>(p.out)[o] = out[i];
        } else if (mine) {
          static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(out[i]);
          if (p.gu_out) {
            __nv_bfloat16* gu =
                reinterpret_cast<__nv_bfloat16*>(p.gu_out) + (row0 + r) * 2 * p.F + cta0 + ch;
            gu[0] = __float2bfloat16_rn(v);
            gu[p.F] = __float2bfloat16_rn(v1);
          }
        }
      }
    }
    if constexpr (kQuant) {
      if constexpr (S > 1) cluster_sync();
      else __syncthreads();
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = tid + i * kThreads, r = at / kChannels, ch = at % kChannels;
        if (8 * kChannels < kThreads && r >= 8) break;
        int m = amax[r];
        if constexpr (S > 1) {
          const uint32_t here = smem_u32(&amax[r]);
#pragma unroll
          for (uint32_t q = 0; q < S; ++q) {
            int v;
            asm volatile("ld.shared::cluster.s32 %0, [%1];"
                         : "=r"(v)
                         : "r"(cluster_addr(here, q))
                         : "memory");
            m = max(m, v);
          }
        }
        const float scale = __fdiv_rn(__int_as_float(m), 448.0f);
        if (r < rows) {
          const int c = cta0 + ch;
          const float q = scale > 0.0f ? __fdiv_rn(out[i], scale) : 0.0f;
          static_cast<uint8_t*>(p.out)[(row0 + r) * p.F + c] =
              (uint8_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
          if ((c & 127) == 0) p.out_scale[(row0 + r) * (p.F >> 7) + (c >> 7)] = scale;
        }
      }
      // read by all before the next pass, or the CTA's end
      if constexpr (S > 1) cluster_sync();
    }
    __syncthreads();
  }
}

template <int OP, int TYPE, int S>
cudaError_t launch(long long grid, const ExpertArgs& p, const void* a, const void* b,
                   cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = OP == kGated && TYPE == kE4m3 && S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_expert_rows<OP, TYPE, S>, p, a, b);
}

template <int OP, int TYPE>
cudaError_t launch(const ExpertArgs& p, const void* a, const void* b, int num_sms,
                   cudaStream_t st) {
  const int channels = OP == kGated ? 16 : 32;  // of a warp
  const long long segments = p.E < p.rows_max ? p.E : p.rows_max;
  const auto ctas = [&](int s) {
    const int c = channels * (kWarps / s);
    return segments * ((p.N + c - 1) / c);
  };
  // The smallest split that still gives three CTAs per SM (us at four / three /
  // two, one token of E = 256, top-8, H = 7168, F = 2048: down e4m3 24.2 / 24.3 /
  // 26.0, gated e4m3 55.8 / 44.4 / 44.2); two where the split's CTAs form clusters, which cost more (E = 64,
  // H = 2048, F = 1024, top-2: 11.7 / 11.2 / 9.6).
  // int8 warps, which keep loading while they convert, need one (the caches empty, means of 150 in
  // turn within 0.1, three / one: gated 51.5 / 48.6, down 30.7 / 28.6; E = 8 of one row each,
  // H = 4096, F = 1408 29.6 / 29.2 and 19.2 / 16.3; E = 64, H = 2048, F = 1024, top-2 the same;
  // two tokens of the first, gated 86.7 / 85.6, but down 47.1 / 51.5).
  const long long enough =
      (TYPE == kInt8 ? 1ll : OP == kGated && TYPE == kE4m3 ? 2ll : 3ll) * num_sms;
  int s = 1;
  while (s < 8 && ctas(s) < enough) s *= 2;
  switch (s) {
    case 1: return launch<OP, TYPE, 1>(ctas(1), p, a, b, st);
    case 2: return launch<OP, TYPE, 2>(ctas(2), p, a, b, st);
    case 4: return launch<OP, TYPE, 4>(ctas(4), p, a, b, st);
    default: return launch<OP, TYPE, 8>(ctas(8), p, a, b, st);
  }
}

}  // namespace

cudaError_t launch_expert_rows(ExpertOp op, ExpertType type, const ExpertArgs& p, const void* a,
                               const void* b, int num_sms, cudaStream_t st) {
  const bool gated = op == kGated;
  switch (type) {
    case kE4m3:
      return gated ? launch<kGated, kE4m3>(p, a, b, num_sms, st)
                   : launch<kDown, kE4m3>(p, a, b, num_sms, st);
    case kInt8:
      return gated ? launch<kGated, kInt8>(p, a, b, num_sms, st)
                   : launch<kDown, kInt8>(p, a, b, num_sms, st);
    default:
      return gated ? launch<kGated, kBf16>(p, a, b, num_sms, st)
                   : launch<kDown, kBf16>(p, a, b, num_sms, st);
  }
}

}  // namespace moe
