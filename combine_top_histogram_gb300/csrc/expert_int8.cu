// expert_int8.cu -- the experts' forward products of int8 codes over the
// receive segments, on the 5th-generation tensor cores.
//
//   kGated  h = silu(g) u,  g = (sum_k x wg) sx swg,  u = (sum_k x wu) sx swu
//   kDown   y = (sum_k h w2) sh sw2
//
// These tensor cores have no 8-bit integer products. An int8 code is exact in
// fp16, a product of two is exact in the fp32 accumulator, and so is every sum
// below 2^24: the codes stay 8 bits wide in memory and on their way to the SM,
// and become fp16 there.
//
// What that costs is shared memory's 128 bytes a cycle: 64 k of a CTA's 256
// channels and 128 tokens are 512 cycles of products. The weights are therefore the A
// operand, which the tensor cores can take from tensor memory: converted codes
// go there straight from registers and use no shared memory again. Tokens are
// the B operand: their fp16 has to be written to shared memory and read by the products.
//
// One persistent CTA per SM (CG = 1), or two that share a tile of tokens
// (CG = 2: each converts half of the tokens, which the products of both read, and
// its own channels). A CTA's tile is two blocks of 128 channels (kGated: gate and
// up of the same ones, kDown: neighbours) by up to 128 tokens:
//   warp 0       copies codes with TMA into a ring of stages (128 k)
//   warp 1       issues the products (CG = 2: of both CTAs; the second CTA's
//                passes on that its operands are ready)
//   warps 4-11   convert: weights to tensor memory, tokens to shared memory, in
//                four buffers of 64 k
//   warps 12-19  read the accumulators (256 columns: with the operand's 256 the
//                tensor memory is full, so there is one pair of them) into
//                registers, hand them back, and scale and store the results
//                beside the next tile's products
// Channels lie along the accumulator's lanes and tokens along its columns, so
// a warp stores 32 neighbouring channels of one token at a time, and a short
// segment shortens everything but the weights: its tokens are copied,
// converted, multiplied and stored 32 at a time (CG = 2: 64).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "expert_internal.cuh"
#include "expert_math.cuh"
#include "expert_ptx.cuh"
#include "expert_walk.cuh"
#include "internal.cuh"

namespace moe {
namespace {

constexpr int kTokens = 128;           // of a tile: columns of an accumulator
constexpr int kBlock = 128;            // channels of a block: lanes of an accumulator
constexpr int kBoxTokens = 32;         // tokens of one copy
constexpr int kThreads = 640;
constexpr int kConvWarp0 = 4, kEpiWarp0 = 12, kWarps = 8;  // 8 warps each
constexpr int kStageK = 128;           // k of a stage, 128 bytes a row
constexpr int kStepK = 64;             // k of an fp16 buffer, 128 bytes a row
constexpr int kSteps = 4;              // fp16 buffers
constexpr int kWeightBytes = 2 * kBlock * kStageK;
constexpr uint32_t kAcc = kTokens;     // tensor-memory columns of an accumulator
constexpr uint32_t kOperand = 256;     // first column of the fp16 weights
constexpr uint32_t kBlockColumns = kStepK / 2, kStepColumns = 2 * kBlockColumns;

// Registers of a thread: the launch's 20 warps x 96, split between the copying
// and issuing warps (4), the converting (8) and the epilogue's (8), which hold 128 sums:
// 4 * 48 + 8 * 64 + 8 * 152 = 20 * 96.
constexpr int kRegisters = 96;

template <int CG>
struct Plan {
  static constexpr int kOwnTokens = kTokens / CG;  // tokens whose codes this CTA converts
  static constexpr int kStageBytes = kWeightBytes + kOwnTokens * kStageK;
  static constexpr int kStages = CG == 1 ? 3 : 4;
  static constexpr int kStepBytes = kOwnTokens * 128;
};
constexpr int kMaxStages = 4;

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t ready[kSteps], used[kSteps];
  uint64_t dfull, dempty, drain;
  float scale[kWarps][64];             // of an epilogue warp's tokens
  uint32_t tmem;
  int abort;
  int off[MOE_MAX_EXPERTS + 1];
  int pre[MOE_MAX_EXPERTS + 1];        // row tiles before expert e
};

template <int CG>
constexpr int smem_bytes() {
  using P = Plan<CG>;
  constexpr int bytes =
      1024 + P::kStages * P::kStageBytes + kSteps * P::kStepBytes + (int)sizeof(Shared);
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  // more than half of an SM's: a second CTA, and with it a second allocation
  // of the tensor memory, never shares it
  static_assert(bytes > 114 * 1024, "one CTA per SM");
  return bytes;
}

// Tokens of a tile that are copied, converted and multiplied: the segment's, up
// to a whole number of copies for each CTA.
template <int CG>
__device__ __forceinline__ int tile_tokens(int rows) {
  constexpr int unit = kBoxTokens * CG;
  return (min(rows, kTokens) + unit - 1) / unit * unit;
}

// A place in a ring of N buffers, and the parity of its phase.
template <int N>
struct Ring {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      phase ^= 1;
    }
  }
};

template <int OP, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    k_expert_int8(const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_w, const ExpertArgs p) {
  using P = Plan<CG>;
  constexpr bool kPair = CG == 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* steps = smem + P::kStages * P::kStageBytes;
  Shared& s = *reinterpret_cast<Shared*>(steps + kSteps * P::kStepBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? (int)(blockIdx.x & 1) : 0;  // clusters are pairs of neighbours

  if (warp == 2) tc_alloc<CG>(smem_u32(&s.tmem), 512);
  if (threadIdx.x == 0) {
    s.abort = 0;
    for (int i = 0; i < P::kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), kWarps);
    }
    for (int i = 0; i < kSteps; ++i) {
      // the converting warps, and in the first CTA of a pair the second one's word
      mbar_init(smem_u32(&s.ready[i]), kWarps + (kPair && rank == 0 ? 1 : 0));
      mbar_init(smem_u32(&s.used[i]), 1);
    }
    mbar_init(smem_u32(&s.dfull), 1);
    mbar_init(smem_u32(&s.dempty), kWarps * CG);
    mbar_init(smem_u32(&s.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_w);
  }
  pdl_wait();  // the segments and the operands come from earlier kernels
  load_segments<kTokens, kThreads>(p, s);
  tc_fence_before();
  if constexpr (kPair) cluster_sync();  // both CTAs' barriers exist
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const WaitCtl ctl{&s.abort, kPair ? cluster_addr(smem_u32(&s.abort), rank ^ 1) : 0u, p.wait_limit,
                    p.status};
  Walk<false, kTokens, Shared> walk(p, s, kStageK, 0, blockIdx.x / CG, gridDim.x / CG);
  const int step_count = (p.K + kStepK - 1) / kStepK;  // of a tile
  // this CTA's first channel within a tile's, and a tile's channels
  constexpr int kOwn = OP == kGated ? kBlock : 2 * kBlock, kAll = kOwn * CG;
  const int own = rank * kOwn;

  if (warp < kConvWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 0) {
      Ring<P::kStages> ring;
      uint32_t announced = 0;
      bool ok = true;
      Tile t;
      while (ok && walk.next(t)) {
        // uniform, and known to be
        const int blocks = __shfl_sync(~0u, t.kb, 0), e = __shfl_sync(~0u, t.e, 0);
        const int n = tile_tokens<CG>(__shfl_sync(~0u, t.rows, 0)) / CG;  // of this CTA
        const int row0 = __shfl_sync(~0u, t.row0, 0) + rank * n;
        const int c0 = __shfl_sync(~0u, t.n0, 0) * kAll + own;
        const uint32_t bytes = kWeightBytes + n * kStageK;
        for (int kb = 0; kb < blocks; ++kb) {
          ok = __all_sync(~0u, mbar_wait<kPair>(smem_u32(&s.empty[ring.i]), ring.phase ^ 1, ctl));
          if (!ok) break;
          const uint32_t bar = smem_u32(&s.full[ring.i]);
          const uint32_t w = smem_u32(smem) + ring.i * P::kStageBytes, x = w + kWeightBytes;
          mbar_expect_elected(bar, bytes);
          tma_load_3d<1>(w, &map_w, bar, kb * kStageK, c0, e);
          tma_load_3d<1>(w + kBlock * kStageK, &map_w, bar, kb * kStageK,
                         OP == kGated ? p.F + c0 : c0 + kBlock, e);
          for (int i = 0; i < n; i += kBoxTokens)
            tma_load_2d<1>(x + i * kStageK, &map_x, bar, kb * kStageK, row0 + i);
          ++announced;
          ring.next();
        }
      }
      // copies in flight land before the CTA ends, also when a wait gave up
      const uint32_t left = announced < P::kStages ? announced : P::kStages;
      for (uint32_t i = announced - left; i != announced; ++i)
        mbar_drain(smem_u32(&s.full[i % P::kStages]), (i / P::kStages) & 1);
      __syncwarp();
    } else if (warp == 1 && rank == 0) {
      Ring<kSteps> ring;
      uint32_t dphase = 1;
      bool ok = true;
      Tile t;
      while (ok && walk.next(t)) {
        const int n = tile_tokens<CG>(__shfl_sync(~0u, t.rows, 0));
        const uint32_t idesc = mma_desc(true, false, false, kBlock * CG, n);
        ok = __all_sync(~0u, mbar_wait<kPair>(smem_u32(&s.dempty), dphase, ctl));
        if (!ok) break;
        dphase ^= 1;
        for (int j = 0; j < step_count; ++j) {
          ok = __all_sync(~0u, mbar_wait<kPair>(smem_u32(&s.ready[ring.i]), ring.phase, ctl));
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = tmem + kOperand + ring.i * kStepColumns;
          const uint64_t b = smem_desc(smem_u32(steps) + ring.i * P::kStepBytes, 16, 1024);
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // 16 k: 8 columns of A, 32 bytes of a row of B
            tc_mma_ta<CG>(tmem, a + 8 * k, b + 2 * k, idesc, j > 0 || k > 0);
            tc_mma_ta<CG>(tmem + kAcc, a + kBlockColumns + 8 * k, b + 2 * k, idesc, j > 0 || k > 0);
          }
          tc_commit<CG>(smem_u32(&s.used[ring.i]));
          ring.next();
        }
        if (ok) tc_commit<CG>(smem_u32(&s.dfull));
      }
      __syncwarp();
      tc_commit<CG>(smem_u32(&s.drain));  // products in flight end before TMEM is freed
      mbar_drain(smem_u32(&s.drain), 0);
      __syncwarp();
    } else if (warp == 1) {
      // the second CTA's operands are ready: a word to the first, whose products read them
      Ring<kSteps> ring;
      bool ok = true;
      Tile t;
      while (ok && walk.next(t)) {
        for (int j = 0; j < step_count; ++j) {
          ok = __all_sync(~0u, mbar_wait<kPair>(smem_u32(&s.ready[ring.i]), ring.phase, ctl));
          if (!ok) break;
          tc_fence_after();
          tc_fence_before();
          if (lane == 0) mbar_arrive_release(cluster_addr(smem_u32(&s.ready[ring.i]), 0));
          __syncwarp();
          ring.next();
        }
      }
      __syncwarp();
    }
  } else if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int cw = warp - kConvWarp0, block = cw >> 2;
    const int row = (warp & 3) * 32 + lane;  // of the weight block: its lane of tensor memory
    const uint32_t to = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kOperand + block * kBlockColumns;
    // token and first 16-byte unit of its 64 k: CG = 1 two units a thread, else one
    const int ct = cw * 32 + lane, token = ct % P::kOwnTokens, unit0 = ct / P::kOwnTokens * (2 / CG);
    Ring<P::kStages> ring;
    Ring<kSteps> step;
    bool ok = true;
    Tile t;
    while (ok && walk.next(t)) {
      const bool mine = token < tile_tokens<CG>(t.rows) / CG;
      for (int j = 0; j < step_count; ++j) {
        const int half = j & 1;  // of the stage
        if (half == 0)
          ok = mbar_wait<kPair>(smem_u32(&s.full[ring.i]), ring.phase, ctl);
        ok = ok && mbar_wait<kPair>(smem_u32(&s.used[step.i]), step.phase ^ 1, ctl);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        tc_fence_after();
        const uint8_t* stage = smem + ring.i * P::kStageBytes;
        const uint4* w = reinterpret_cast<const uint4*>(stage + (block * kBlock + row) * kStageK);
        const uint4* x = reinterpret_cast<const uint4*>(stage + kWeightBytes + token * kStageK);
        uint4* out = reinterpret_cast<uint4*>(steps + step.i * P::kStepBytes + token * 128);
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // 32 k of the weights
          uint32_t v[16];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint4 c = w[(half * 4 + 2 * i + u) ^ (row & 7)];
            const uint32_t cc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint2 f = int8_to_f16(cc[q]);
              v[8 * u + 2 * q] = f.x;
              v[8 * u + 2 * q + 1] = f.y;
            }
          }
          tc_st16(to + step.i * kStepColumns + 16 * i, v);
        }
        if (mine) {
#pragma unroll
          for (int i = 0; i < 2 / CG; ++i) {  // 16 k of a token: 32 bytes of fp16
            const int u = unit0 + i;
            const uint4 c = x[(half * 4 + u) ^ (token & 7)];
            const uint2 f0 = int8_to_f16(c.x), f1 = int8_to_f16(c.y), f2 = int8_to_f16(c.z),
                        f3 = int8_to_f16(c.w);
            out[(2 * u) ^ (token & 7)] = make_uint4(f0.x, f0.y, f1.x, f1.y);
            out[(2 * u + 1) ^ (token & 7)] = make_uint4(f2.x, f2.y, f3.x, f3.y);
          }
        }
        tc_wait_st();
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&s.ready[step.i]));
          if (half == 1 || j == step_count - 1) mbar_arrive(smem_u32(&s.empty[ring.i]));
        }
        if (half == 1 || j == step_count - 1) ring.next();
        step.next();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
    const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + half * 64;
    uint32_t dphase = 0;
    bool ok = true;
    Tile t;
    while (ok && walk.next(t)) {
      const int left = t.rows - half * 64;  // tokens of this warp: columns half * 64 on
      const int c = t.n0 * kAll + own + quarter * 32 + lane;  // channel, of the first block
      const int c1 = OP == kGated ? c + p.F : c + kBlock;
      const int channels = OP == kGated ? 2 * p.F : p.N;
      const bool in0 = c < p.N, in1 = OP == kGated ? in0 : c1 < p.N;
      const float* sw = p.sb + (long long)t.e * channels;
      const float w0 = in0 ? __ldg(sw + c) : 0.0f, w1 = in1 ? __ldg(sw + c1) : 0.0f;
      const float* sx = p.sa + t.row0 + half * 64;
      float* scale = s.scale[warp - kEpiWarp0];
#pragma unroll
      for (int i = 0; i < 64; i += 32) scale[lane + i] = lane + i < left ? __ldg(sx + lane + i) : 0.0f;
      ok = __all_sync(~0u, mbar_wait<kPair>(smem_u32(&s.dfull), dphase, ctl));
      if (!ok) break;
      dphase ^= 1;
      tc_fence_after();
      uint32_t v[4][32];  // first block's 64 columns, then the second's
#pragma unroll
      for (int q = 0; q < 4; ++q) tc_ld32(v[q], from + (q & 1) * 32 + (q >> 1) * kAcc);
      tc_wait_ld();
#pragma unroll
      for (int q = 0; q < 4; ++q) tc_loaded(v[q]);
      tc_fence_before();
      __syncwarp();  // the scales are written, too
      if (lane == 0) {
        if constexpr (kPair) mbar_arrive_relaxed(cluster_addr(smem_u32(&s.dempty), 0));
        else mbar_arrive(smem_u32(&s.dempty));
      }
      // one token after the other: of 32 neighbouring channels a warp writes 128 bytes of h, or 64
      // of y in each block
      using Out = std::conditional_t<OP == kGated, float, __nv_bfloat16>;
      Out* out = static_cast<Out*>(p.out) + ((long long)t.row0 + half * 64) * p.N + c;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (left > q * 16) {
#pragma unroll
          for (int i = q * 16; i < q * 16 + 16; ++i) {
            const float sr = scale[i];
            const float a = __uint_as_float(v[i >> 5][i & 31]) * sr * w0;
            const float b = __uint_as_float(v[2 + (i >> 5)][i & 31]) * sr * w1;
            if constexpr (OP == kGated) {
              if (in0 && i < left) *out = silu(a) * b;
            } else {
              if (in0 && i < left) *out = __float2bfloat16_rn(a);
              if (in1 && i < left) out[kBlock] = __float2bfloat16_rn(b);
            }
            out += p.N;
          }
        }
      }
      __syncwarp();  // read, before the next tile's are written
    }
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (kPair) cluster_sync();  // neither CTA's memory is used any more
  else __syncthreads();
  tc_fence_after();
  if (warp == 2) tc_dealloc<CG>(tmem, 512);
}

// ---- host side -------------------------------------------------------------
template <int OP, int CG>
cudaError_t launch(const ExpertArgs& args, const void* a, const void* b, int num_sms,
                   cudaStream_t st) {
  ExpertArgs p = args;
  constexpr int channels = (OP == kGated ? kBlock : 2 * kBlock) * CG;
  p.nt = (p.N + channels - 1) / channels;
  CUtensorMap mx, mw;
  cudaError_t e = make_map(&mx, a, true, p.K, p.rows_max, 0, kBoxTokens);
  if (e == cudaSuccess)
    e = make_map(&mw, b, true, p.K, OP == kGated ? 2ll * p.F : p.N, p.E, kBlock);
  if (e != cudaSuccess) return e;
  const long long segments = p.E < p.rows_max ? p.E : p.rows_max;
  const long long tiles = (p.rows_max / kTokens + segments) * p.nt, most = num_sms / CG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<CG>();
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_expert_int8<OP, CG>, mx, mw, p);
}

template <int OP, int CG>
cudaError_t prepare() {
  const auto kernel = k_expert_int8<OP, CG>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem_bytes<CG>());
  if (e != cudaSuccess) return e;
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return e;
  return attr.numRegs >= kRegisters ? cudaSuccess : cudaErrorInvalidConfiguration;
}

}  // namespace

cudaError_t expert_int8_prepare() {
  cudaError_t e = prepare<kGated, 1>();
  if (e == cudaSuccess) e = prepare<kDown, 1>();
  return e;
}

cudaError_t launch_expert_int8(ExpertOp op, const ExpertArgs& p, const void* a, const void* b,
                               int num_sms, cudaStream_t st) {
  return op == kGated ? launch<kGated, 1>(p, a, b, num_sms, st)
                      : launch<kDown, 1>(p, a, b, num_sms, st);
}

}  // namespace moe
