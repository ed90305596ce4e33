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
// The conversions are what bounds a tile. The weights are the A operand, which the
// tensor cores take from tensor memory: as fp16 in shared memory they would be
// stored there and read again. A step of 64 k and n tokens, whose products with 256
// channels take 4 n cycles, is
//   weights (A)  16 KB of codes in and out of shared memory, 32 KB of fp16 to tensor memory
//   tokens (B)   64 n bytes in and out, 128 n of fp16 to shared memory
// beside the 256 n that the products read. The weights' part is the same for any n,
// so n is as large as tensor memory allows: 192, where 384 columns of accumulators
// and 128 of weights fill it. Their 768 cycles of products then take 1010 to 1030 (by the
// clocks of the issuing warp; 940 at 128 tokens, 830 to 870 at 64); the
// vector pipes are 60-70 % busy by then, instruction issue 50-67 %, and the warps wait
// on stores to tensor and shared memory in turn. Gated, E = 64, 512 rows each, H = 7168,
// F = 2048: 1310 to 1340 us a call on its own, 1.44 PFLOP/s, 0.77 of the measured fp16 rate, and
// 1510 back to back, where the power limit lowers the clock; products of many rows
// an expert are widened in memory first (expert_codes.cu).
//
// One persistent CTA per SM, or, where tiles are few and the reduction is long, a
// cluster of CTAs for each tile (SPLIT, below). A tile is two blocks of 128 channels
// (kGated: gate and up of the same ones, kDown: neighbours) by up to 192 tokens:
//   warps 0, 3   copy codes with TMA into rings of stages, of weights (128 k) and of
//                tokens (64 k)
//   warp 1       issues the products, a step of 64 k at a time
//   warps 4-19   convert: weights to slots of tensor memory, tokens to buffers of fp16
//                in shared memory; eight warps take every other step, so that one step's
//                loads, conversions and stores run beside the next one's
//   warps 20-27  read the accumulators 32 tokens at a time, scale and store them; with
//                the last of them read the accumulators are handed back
// Steps of 64 k and not 32 halve the waits and hand-overs of a tile (the case above, on
// its own: 1590 us with 32).
// Channels lie along the accumulator's lanes and tokens along its columns, so
// a warp stores 32 neighbouring channels of one token at a time, and a short
// segment shortens everything but the weights: its tokens are copied,
// converted, multiplied and stored 32 at a time.
// Of tiles with fewer tokens, those of 128 convert ahead into four slots, those of 64
// into six: few rows an expert are bound by the weights' bytes (gated, E = 256, 32 rows
// each: 1360 us, 0.83 of the copy rate).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "expert_internal.cuh"
#include "expert_math.cuh"
#include "expert_ptx.cuh"
#include "expert_walk.cuh"
#include "internal.cuh"

namespace moe {
namespace {

constexpr int kBlock = 128;            // channels of a block: lanes of an accumulator
constexpr int kConvWarp0 = 4, kConvWarps = 16, kEpiWarp0 = 20, kEpiWarps = 8;
constexpr int kThreads = 896;
constexpr int kStageK = 128;           // k of a stage of weights, 128 bytes a row
constexpr int kStepK = 64;             // k of a step and of a stage of tokens, 64 bytes a row
constexpr int kWBytes = 2 * kBlock * kStageK;
constexpr uint32_t kBlockColumns = kStepK / 2, kStepColumns = 2 * kBlockColumns;
constexpr int kMaxTokens = 192, kMaxRing = 6;

// TOKENS of a tile; SLOTS of the tensor memory for a step's fp16 weights;
// stages of codes of weights and tokens; BUFFERS of a step's fp16 tokens; BOX:
// tokens of one copy.
template <int TOKENS, int SLOTS, int W_STAGES, int X_STAGES, int BUFFERS, int BOX>
struct Plan {
  // of the largest tiles, shared memory has room for no more experts' segments
  static constexpr int kExperts = TOKENS == 192 ? 768 : MOE_MAX_EXPERTS;
  // the second half of a step's weights is converted after the slot is free: a few
  // more cycles there, but registers for the rest where a thread has two tokens or three
  static constexpr bool kSplit = TOKENS > 64;
  static constexpr int kTokens = TOKENS, kSlots = SLOTS, kBuffers = BUFFERS, kBox = BOX;
  static constexpr int kWStages = W_STAGES, kXStages = X_STAGES;
  static constexpr int kXBytes = kTokens * kStepK, kBufferBytes = kTokens * 2 * kStepK;
  static constexpr uint32_t kAcc = kTokens;       // tensor-memory columns of an accumulator
  static constexpr uint32_t kOperand = 2 * kAcc;  // first column of the fp16 weights
  static constexpr int kRingBytes =
      kWStages * kWBytes + kXStages * kXBytes + kBuffers * kBufferBytes;
  static_assert(2 * kTokens * kBlock * 4 <= kRingBytes, "a split tile's sums");
  static_assert(kOperand + kSlots * kStepColumns <= 512, "tensor memory");
  static_assert(kWStages <= kMaxRing && kXStages <= kMaxRing && kSlots <= kMaxRing &&
                kBuffers <= kMaxRing, "");
  static_assert(kTokens <= kMaxTokens && kTokens % 64 == 0 && kTokens % kBox == 0 &&
                kXBytes % 1024 == 0, "");
};
using Many = Plan<192, 2, 3, 4, 3, 64>;
using Some = Plan<128, 4, 3, 6, 3, 64>;
using Few = Plan<64, 6, 4, 4, 4, 32>;

// Registers of a thread: the launch's 28 warps x 72, split between the copying
// and issuing warps (4), the converting (16) and the epilogue's (8), which hold
// 64 sums at a time: 4 * 40 + 16 * 64 + 8 * 104 = 28 * 72.
constexpr int kRegisters = 72;

template <class P>
struct Shared {
  uint64_t wfull[kMaxRing], wempty[kMaxRing], xfull[kMaxRing], xempty[kMaxRing];
  uint64_t ready[kMaxRing], used[kMaxRing], xused[kMaxRing];
  uint64_t dfull, dempty, drain;
  float scale[kEpiWarps][P::kTokens / 2];  // of an epilogue warp's tokens
  uint32_t tmem;
  int abort;
  int off[P::kExperts + 1];
  int pre[P::kExperts + 1];            // row tiles before expert e
};

template <class P>
constexpr int smem_bytes() {
  constexpr int bytes = 1024 + P::kRingBytes + (int)sizeof(Shared<P>);
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  // more than half of an SM's: a second CTA, and with it a second allocation
  // of the tensor memory, never shares it
  static_assert(bytes > 114 * 1024, "one CTA per SM");
  return bytes;
}

// Tokens of a tile that are converted and multiplied.
template <class P>
__device__ __forceinline__ int tile_tokens(int rows) {
  return (min(rows, P::kTokens) + 31) / 32 * 32;
}

// All lanes wait for the phase of the given parity; false when a wait gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl& ctl) {
  if (__all_sync(~0u, mbar_test(bar, parity))) return true;
  return __all_sync(~0u, mbar_wait<false>(bar, parity, ctl));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// A store under a predicate, without a branch around it.
__device__ __forceinline__ void store_if(void* p, uint32_t v, bool ok) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q st.global.b32 [%0], %1;\n\t}" ::"l"(
                   p),
               "r"(v), "r"((int)ok)
               : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t*>(&v);
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
  __device__ __forceinline__ void skip() {  // to the next but one
    i += 2;
    if (i >= N) {
      i -= N;
      phase ^= 1;
    }
  }
  __device__ __forceinline__ void back() {
    if (--i < 0) {
      i = N - 1;
      phase ^= 1;
    }
  }
};

// Waits for the copies of the last `announced` stages of a ring, of as many as it has.
template <int N>
__device__ __forceinline__ void drain_ring(const uint64_t* full, uint32_t announced) {
  const uint32_t left = announced < N ? announced : N;
  for (uint32_t i = announced - left; i != announced; ++i)
    mbar_drain(smem_u32(&full[i % N]), (i / N) & 1);
}

// SPLIT: a cluster takes one tile, each of its CTAs a share of the reduction axis. Their sums
// meet in shared memory and are added up in the order of the ranks, a rank for every so many
// tokens.
template <int OP, class P, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    k_expert_int8(const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_w, const ExpertArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* wring = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* xring = wring + P::kWStages * kWBytes;
  uint8_t* buffers = xring + P::kXStages * P::kXBytes;
  Shared<P>& s = *reinterpret_cast<Shared<P>*>(wring + P::kRingBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 2) tc_alloc<1>(smem_u32(&s.tmem), 512);
  if (threadIdx.x == 0) {
    s.abort = 0;
    for (int i = 0; i < P::kWStages; ++i) {
      mbar_init(smem_u32(&s.wfull[i]), 1);
      mbar_init(smem_u32(&s.wempty[i]), kConvWarps);
    }
    for (int i = 0; i < P::kXStages; ++i) {
      mbar_init(smem_u32(&s.xfull[i]), 1);
      mbar_init(smem_u32(&s.xempty[i]), kConvWarps / 2);
    }
    for (int i = 0; i < P::kSlots; ++i) {
      mbar_init(smem_u32(&s.ready[i]), kConvWarps / 2);
      mbar_init(smem_u32(&s.used[i]), 1);
    }
    for (int i = 0; i < P::kBuffers; ++i) mbar_init(smem_u32(&s.xused[i]), 1);
    mbar_init(smem_u32(&s.dfull), 1);
    mbar_init(smem_u32(&s.dempty), kEpiWarps);
    mbar_init(smem_u32(&s.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_w);
  }
  pdl_wait();  // the segments and the operands come from earlier kernels
  load_segments<P::kTokens, kThreads>(p, s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const WaitCtl ctl{&s.abort, 0u, p.wait_limit, p.status};
  const int ranks = SPLIT ? (int)cluster_size() : 1;
  const int rank = SPLIT ? (int)blockIdx.x % ranks : 0;
  Walk<false, P::kTokens, Shared<P>> walk(p, s, kStageK, 0, blockIdx.x / ranks, gridDim.x / ranks);
  // of a tile, this CTA's stages of weights and steps
  const int stages = (p.K + kStageK - 1) / kStageK, stage0 = stages * rank / ranks,
            stage1 = stages * (rank + 1) / ranks;
  const int step0 = 2 * stage0, step_count = min(2 * stage1, (p.K + kStepK - 1) / kStepK) - step0;
  constexpr int kChannels = OP == kGated ? kBlock : 2 * kBlock;  // a tile's output channels

  if (warp < kConvWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {  // weights
      Ring<P::kWStages> ring;
      uint32_t announced = 0;
      bool ok = true;
      Tile t;
      while (ok && walk.next(t)) {
        // uniform, and known to be
        const int e = __shfl_sync(~0u, t.e, 0);
        const int c0 = __shfl_sync(~0u, t.n0, 0) * kChannels;
        const int c1 = OP == kGated ? p.F + c0 : c0 + kBlock;
        for (int kb = stage0; kb < stage1; ++kb) {
          ok = __all_sync(~0u, mbar_wait<false>(smem_u32(&s.wempty[ring.i]), ring.phase ^ 1, ctl));
          if (!ok) break;
          const uint32_t bar = smem_u32(&s.wfull[ring.i]), w = smem_u32(wring) + ring.i * kWBytes;
          mbar_expect_elected(bar, kWBytes);
          tma_load_3d<1>(w, &map_w, bar, kb * kStageK, c0, e);
          tma_load_3d<1>(w + kBlock * kStageK, &map_w, bar, kb * kStageK, c1, e);
          ++announced;
          ring.next();
        }
        if (SPLIT) break;
      }
      // copies in flight land before the CTA ends, also when a wait gave up
      drain_ring<P::kWStages>(s.wfull, announced);
      __syncwarp();
    } else if (warp == 3) {  // tokens
      Ring<P::kXStages> ring;
      uint32_t announced = 0;
      bool ok = true;
      Tile t;
      while (ok && walk.next(t)) {
        const int row0 = __shfl_sync(~0u, t.row0, 0);
        const int n = tile_tokens<P>(__shfl_sync(~0u, t.rows, 0)), copies = (n + P::kBox - 1) / P::kBox;
        for (int j = 0; j < step_count; ++j) {
          ok = __all_sync(~0u, mbar_wait<false>(smem_u32(&s.xempty[ring.i]), ring.phase ^ 1, ctl));
          if (!ok) break;
          const uint32_t bar = smem_u32(&s.xfull[ring.i]), x = smem_u32(xring) + ring.i * P::kXBytes;
          mbar_expect_elected(bar, copies * P::kBox * kStepK);
          for (int i = 0; i < copies; ++i)
            tma_load_2d<1>(x + i * P::kBox * kStepK, &map_x, bar, (step0 + j) * kStepK,
                           row0 + i * P::kBox);
          ++announced;
          ring.next();
        }
        if (SPLIT) break;
      }
      drain_ring<P::kXStages>(s.xfull, announced);
      __syncwarp();
    } else if (warp == 1) {
      Ring<P::kSlots> slot;
      Ring<P::kBuffers> buffer;
      uint32_t dphase = 1;
      bool ok = true;
      Tile t;
      while (ok && walk.next(t)) {
        const uint32_t idesc =
            mma_desc(true, false, false, kBlock, tile_tokens<P>(__shfl_sync(~0u, t.rows, 0)));
        ok = __all_sync(~0u, mbar_wait<false>(smem_u32(&s.dempty), dphase, ctl));
        if (!ok) break;
        dphase ^= 1;
        for (int j = 0; j < step_count; ++j) {
          ok = __all_sync(~0u, mbar_wait<false>(smem_u32(&s.ready[slot.i]), slot.phase, ctl));
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = tmem + P::kOperand + slot.i * kStepColumns;
          const uint64_t b = smem_desc(smem_u32(buffers) + buffer.i * P::kBufferBytes, 16, 1024);
#pragma unroll
          for (int k = 0; k < kStepK / 16; ++k) {  // 16 k: 8 columns of A, 32 bytes of a row of B
            tc_mma_ta(tmem, a + 8 * k, b + 2 * k, idesc, j > 0 || k > 0);
            tc_mma_ta(tmem + P::kAcc, a + kBlockColumns + 8 * k, b + 2 * k, idesc, j > 0 || k > 0);
          }
          tc_commit<1>(smem_u32(&s.used[slot.i]));
          tc_commit<1>(smem_u32(&s.xused[buffer.i]));
          slot.next();
          buffer.next();
        }
        if (ok) tc_commit<1>(smem_u32(&s.dfull));
        if (SPLIT) break;
      }
      __syncwarp();
      tc_commit<1>(smem_u32(&s.drain));  // products in flight end before TMEM is freed
      mbar_drain(smem_u32(&s.drain), 0);
      __syncwarp();
    }
    if (SPLIT) cluster_sync();  // the sums are written, as for the other warps
  } else if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int cw = warp - kConvWarp0, group = cw >> 3, block = (cw >> 2) & 1;
    const int row = (warp & 3) * 32 + lane;  // of the weight block: its lane of tensor memory
    const uint32_t to =
        tmem + ((uint32_t)((warp & 3) * 32) << 16) + P::kOperand + block * kBlockColumns;
    const int ct = (cw & 7) * 32 + lane;     // thread of the group
    // A step's 16-byte units: four of this thread's channel, and of the tokens those
    // numbered ct + 256 i, all first units before all second ones and so on. The
    // copies leave unit u of a weight row at u ^ (row & 7) of its 128 bytes, and of a token at
    // u ^ (token / 2 & 3) of its 64; the products want unit u of a token's fp16 at u ^ (token & 7).
    constexpr int kPer = P::kTokens * 4 / 256;
    const uint32_t w0 = smem_u32(wring) + (block * kBlock + row) * kStageK +
                        (((group * 4) ^ (row & 7)) << 4);
    uint32_t x0[kPer], o0[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int unit = (ct + 256 * i) / P::kTokens, token = (ct + 256 * i) % P::kTokens;
      x0[i] = smem_u32(xring) + token * 64 + ((unit ^ (token >> 1 & 3)) << 4);
      o0[i] = smem_u32(buffers) + token * 128 + (((2 * unit) ^ (token & 7)) << 4);
    }
    Ring<P::kWStages> wr;
    // this group's next step
    Ring<P::kXStages> xr;
    Ring<P::kBuffers> buffer;
    Ring<P::kSlots> slot;
    if (group == 1) {
      xr.next();
      buffer.next();
      slot.next();
    }
    bool ok = true;
    Tile t;
    while (ok && walk.next(t)) {
      bool mine[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        mine[i] = (ct + 256 * i) % P::kTokens < tile_tokens<P>(t.rows);
      for (int j0 = 0; j0 < step_count; j0 += 2) {
        if (j0 + group < step_count) {
          // 16 k of a token: 32 bytes of fp16
          ok = warp_wait(smem_u32(&s.xfull[xr.i]), xr.phase, ctl);
          if (!ok) break;
          uint4 c[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (mine[i]) c[i] = lds128(x0[i] + xr.i * P::kXBytes);
          ok = warp_wait(smem_u32(&s.xused[buffer.i]), buffer.phase ^ 1, ctl);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            if (mine[i]) {
              const uint2 f0 = int8_to_f16(c[i].x), f1 = int8_to_f16(c[i].y),
                          f2 = int8_to_f16(c[i].z), f3 = int8_to_f16(c[i].w);
              const uint32_t o = o0[i] + buffer.i * P::kBufferBytes;
              sts128(o, make_uint4(f0.x, f0.y, f1.x, f1.y));
              sts128(o ^ 16, make_uint4(f2.x, f2.y, f3.x, f3.y));
            }
          }
          // 64 k of a channel
          ok = warp_wait(smem_u32(&s.wfull[wr.i]), wr.phase, ctl);
          if (!ok) break;
          const uint32_t w = w0 + wr.i * kWBytes;
          uint32_t v[2][16];
          const auto widen = [&](int half) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint4 q = lds128(w ^ (32 * half + 16 * u));
              const uint32_t cc[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                const uint2 f = int8_to_f16(cc[b]);
                v[half][u * 8 + 2 * b] = f.x;
                v[half][u * 8 + 2 * b + 1] = f.y;
              }
            }
          };
          widen(0);
          if (!P::kSplit) widen(1);
          ok = warp_wait(smem_u32(&s.used[slot.i]), slot.phase ^ 1, ctl);
          if (!ok) break;
          tc_fence_after();
          tc_st16(to + slot.i * kStepColumns, v[0]);
          if (P::kSplit) widen(1);
          tc_st16(to + slot.i * kStepColumns + 16, v[1]);
          fence_async_smem();
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_u32(&s.ready[slot.i]));
            mbar_arrive(smem_u32(&s.xempty[xr.i]));
          }
          xr.skip();
          buffer.skip();
          slot.skip();
        } else {  // an odd last step: the other group's
          ok = warp_wait(smem_u32(&s.wfull[wr.i]), wr.phase, ctl);
          if (!ok) break;
        }
        if (lane == 0) mbar_arrive(smem_u32(&s.wempty[wr.i]));
        wr.next();
      }
      // an odd number of steps: each group took every other one up to the last, so the first one's
      // next is one too far and the second's one short
      if (step_count & 1) {
        if (group == 0) {
          xr.back();
          buffer.back();
          slot.back();
        } else {
          xr.next();
          buffer.next();
          slot.next();
        }
      }
      if (SPLIT) break;
    }
    if (SPLIT) cluster_sync();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    constexpr int kHalf = P::kTokens / 2;  // tokens of a warp
    const int quarter = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + half * kHalf;
    float* scale = s.scale[warp - kEpiWarp0];
    uint32_t dphase = 0;
    bool ok = true;
    Tile t;
    t.rows = 0;
    while (ok && walk.next(t)) {
      const int left = t.rows - half * kHalf;  // tokens of this warp: columns half * kHalf on
      const int c = t.n0 * kChannels + quarter * 32 + lane;  // channel, of the first block
      const int c1 = OP == kGated ? c + p.F : c + kBlock;
      const int channels = OP == kGated ? 2 * p.F : p.N;
      const bool in0 = c < p.N, in1 = OP == kGated ? in0 : c1 < p.N;
      const float* sw = p.sb + (long long)t.e * channels;
      const float w0 = in0 ? __ldg(sw + c) : 0.0f, w1 = in1 ? __ldg(sw + c1) : 0.0f;
      const float* sx = p.sa + t.row0 + half * kHalf;
#pragma unroll
      for (int i = 0; i < kHalf; i += 32) scale[lane + i] = lane + i < left ? __ldg(sx + lane + i) : 0.0f;
      ok = __all_sync(~0u, mbar_wait<false>(smem_u32(&s.dfull), dphase, ctl));
      if (!ok) break;
      dphase ^= 1;
      tc_fence_after();
      if (SPLIT) {
        // all copies have landed and all products are done: the rings are free
        float* sums = reinterpret_cast<float*>(wring) + quarter * 32 + lane;
#pragma unroll 1
        for (int i = half * kHalf; i < min(t.rows, (half + 1) * kHalf); i += 32) {
          uint32_t a[32];
#pragma unroll
          for (int blk = 0; blk < 2; ++blk) {
            tc_ld32(a, from - half * kHalf + blk * P::kAcc + i);
            tc_wait_ld();
            tc_loaded(a);
#pragma unroll
            for (int j = 0; j < 32; ++j)
              sums[(blk * P::kTokens + i + j) * kBlock] = __uint_as_float(a[j]);
          }
        }
        break;
      }
      // Rounds of 32 tokens: all values, then all stores. A store before another token's value
      // would hold that one's scale, which the compiler cannot tell from what is stored, until the
      // first is done (gated, E = 19, 576 rows each, H = 1024, F = 2048: 142 / 135 us).
      using Out = std::conditional_t<OP == kGated, float, __nv_bfloat16>;
      const int odd = OP == kGated ? 0 : lane & 1;
      Out* out = static_cast<Out*>(p.out) + ((long long)t.row0 + half * kHalf + odd) * p.N + c - odd;
      const int rounds = left <= 0 ? 0 : min((left + 31) / 32, kHalf / 32);
      __syncwarp();  // the scales are written
#pragma unroll 1
      for (int q = 0; q < rounds; ++q) {
        uint32_t a[32], b[32];  // 32 tokens of the first block, and of the second
        tc_ld32(a, from + q * 32);
        tc_ld32(b, from + P::kAcc + q * 32);
        tc_wait_ld();
        tc_loaded(a);
        tc_loaded(b);
        if (q == rounds - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.dempty));
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float sr = scale[q * 32 + i];
          const float f = __uint_as_float(a[i]) * sr * w0, g = __uint_as_float(b[i]) * sr * w1;
          if constexpr (OP == kGated) {
            a[i] = __float_as_uint(silu(f) * g);
          } else {
            a[i] = __float_as_uint(f);
            b[i] = __float_as_uint(g);
          }
        }
        if constexpr (OP == kGated) {  // 32 channels of a token: 128 bytes
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            store_if(out, a[i], in0 && q * 32 + i < left);
            out += p.N;
          }
        } else {
          // Two tokens at a time: neighbouring lanes exchange theirs, and each holds two channels of
          // one token (32 channels: 64 bytes of each of the two)
          const uint32_t sel = odd ? 0x3276u : 0x5410u;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const bool in = q * 32 + i + odd < left;
            const uint32_t pa = bf16x2(a[i], a[i + 1]), pb = bf16x2(b[i], b[i + 1]);
            store_if(out, __byte_perm(pa, __shfl_xor_sync(~0u, pa, 1), sel), in0 && in);
            store_if(out + kBlock, __byte_perm(pb, __shfl_xor_sync(~0u, pb, 1), sel), in1 && in);
            out += 2ll * p.N;
          }
        }
      }
      if (rounds == 0 && lane == 0) mbar_arrive(smem_u32(&s.dempty));
      __syncwarp();  // read, before the next tile's are written
    }
    if (SPLIT) {
      cluster_sync();
      if (ok && t.rows > 0) {
        const uint32_t sums = smem_u32(wring) + (quarter * 32 + lane) * 4;
        const int c = t.n0 * kChannels + quarter * 32 + lane;
        const int c1 = OP == kGated ? c + p.F : c + kBlock;
        const int channels = OP == kGated ? 2 * p.F : p.N;
        const bool in0 = c < p.N, in1 = OP == kGated ? in0 : c1 < p.N;
        const float* sw = p.sb + (long long)t.e * channels;
        const float w0 = in0 ? __ldg(sw + c) : 0.0f, w1 = in1 ? __ldg(sw + c1) : 0.0f;
        for (int i = rank * 2 + half; i < min(t.rows, P::kTokens); i += 2 * ranks) {
          const float sr = __ldg(p.sa + t.row0 + i);
          float f = 0.0f, g = 0.0f;
#pragma unroll 4
          for (int r = 0; r < ranks; ++r) {
            const uint32_t at = cluster_addr(sums + i * kBlock * 4, r);
            f += ld_cluster(at);
            g += ld_cluster(at + P::kTokens * kBlock * 4);
          }
          f = f * sr * w0;
          g = g * sr * w1;
          const long long o = ((long long)t.row0 + i) * p.N + c;
          if constexpr (OP == kGated) {
            if (in0) static_cast<float*>(p.out)[o] = silu(f) * g;
          } else {
            if (in0) static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(f);
            if (in1) static_cast<__nv_bfloat16*>(p.out)[o + kBlock] = __float2bfloat16_rn(g);
          }
        }
      }
    }
  }
  if (SPLIT) cluster_sync();  // the sums have been read
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tc_dealloc<1>(tmem, 512);
}

// ---- host side -------------------------------------------------------------
template <int OP, class P>
cudaError_t launch(const ExpertArgs& args, const void* a, const void* b, int split, int num_sms,
                   cudaStream_t st) {
  ExpertArgs p = args;
  constexpr int channels = OP == kGated ? kBlock : 2 * kBlock;
  p.nt = (p.N + channels - 1) / channels;
  CUtensorMap mx, mw;
  cudaError_t e = make_map(&mx, a, true, p.K, p.rows_max, 0, P::kBox, kStepK);
  if (e == cudaSuccess)
    e = make_map(&mw, b, true, p.K, OP == kGated ? 2ll * p.F : p.N, p.E, kBlock);
  if (e != cudaSuccess) return e;
  const long long segments = p.E < p.rows_max ? p.E : p.rows_max;
  const long long tiles = (p.rows_max / P::kTokens + segments) * p.nt;
  if (split == 1)
    return launch_pdl(k_expert_int8<OP, P, false>,
                      dim3((unsigned)(tiles < num_sms ? tiles : num_sms)), dim3(kThreads),
                      smem_bytes<P>(), st, mx, mw, p);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split));  // a cluster for each tile that there can be
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<P>();
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_expert_int8<OP, P, true>, mx, mw, p);
}

template <class P>
cudaError_t launch(ExpertOp op, const ExpertArgs& p, const void* a, const void* b, int split,
                   int num_sms, cudaStream_t st) {
  return op == kGated ? launch<kGated, P>(p, a, b, split, num_sms, st)
                      : launch<kDown, P>(p, a, b, split, num_sms, st);
}

template <int OP, class P, bool SPLIT>
cudaError_t prepare() {
  const auto kernel = k_expert_int8<OP, P, SPLIT>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<P>());
  if (e != cudaSuccess) return e;
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return e;
  return attr.numRegs >= kRegisters ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <class P>
cudaError_t prepare() {
  cudaError_t e = prepare<kGated, P, false>();
  if (e == cudaSuccess) e = prepare<kGated, P, true>();
  if (e == cudaSuccess) e = prepare<kDown, P, false>();
  if (e == cudaSuccess) e = prepare<kDown, P, true>();
  return e;
}

}  // namespace

cudaError_t expert_int8_prepare() {
  cudaError_t e = prepare<Many>();
  if (e == cudaSuccess) e = prepare<Some>();
  if (e == cudaSuccess) e = prepare<Few>();
  return e;
}

// The plan and the split with the least turns of the SMs x time of a full tile (a step of one at
// 64 / 128 / 192 tokens: 0.43 / 0.47 / 0.51 us, 850 / 940 / 1020 cycles at 2 GHz). An
// expert's weights are converted once for each of its tiles, so a tile should hold most
// experts' rows; where tiles are few, small ones spread over more SMs. The host knows the rows and the experts,
// and takes the rows of one to be within two standard deviations of a random
// choice of the experts. us of Few / Some / Many (here and below of calls on their own, the
// caches empty, means of 20 to 60 of each in turn, standard errors 1.3 us at most), gated,
// H = 7168, F = 2048,
// random rows of E = 64: 56 on average 418 / 391 / 398, 96 718 / 407 / 426, 112
// 720 / 467 / 443, 160 1061 / 794 / 472, 256 1565 / 955 / 892, 512 2922 / 1733 /
// 1317, E = 256: 32 1365 / 1432 / 1458; down, E = 1, 1024 rows 53 / 45 / 49; gated, E = 8,
// H = 1024, F = 512, 512 rows 29 / 23 / 25. What it gives away: experts of very
// unlike rows.
// Where tiles leave SMs without work, clusters of 2, 4 or 8 CTAs share the reduction of one;
// meeting costs them up to 10 us more. us of one CTA / clusters of 2 / 4 / 8, tiles of 64
// unless said otherwise (standard errors 0.1 at most): down, E = 1, 64 rows, H = 4096,
// F = 14336 (16 tiles) 106.3 / 63.3 / 38.4 / 46.3, H = 7168, F = 2048 (28) 22.7 / 22.4 / 18.3 /
// 32.6; gated, E = 1, 64 rows, H = 4096, F = 2048 (16) 39.4 / 32.0 / 23.1 / 31.5, E = 7, 240
// rows, H = 5488, F = 256 (14) 49.4 / 35.3 / 25.1 / 23.1, E = 8, 200 rows, H = 4096,
// F = 1408 (88) 39.8 / 51.6 / 51.7 / 81.7; down, E = 2, 300 rows, H = F = 4096, tiles of 192
// (32) 42.9 / 38.4 / 26.5 / 54.0. Where they come near one another the rule may miss the
// least: gated, E = 4, 400 rows, H = 1024, F = 512 it takes 18.9 / 21.2 / 18.0 (8 stages: no
// clusters of 8) without clusters, E = 3, 450 rows, H = 4112, F = 400 tiles of 192 in clusters of
// 8, 26.9, where tiles of 64 in clusters of 4 take 24.9. Clusters of 8 have room on 14 x 8 SMs
// only, of 4 on 36 x 4: parts of the GPU have other numbers of SMs.
struct Choice {
  double us;
  int split;
};

template <class P>
static Choice choose(ExpertOp op, const ExpertArgs& p, int num_sms, double step) {
  Choice best{HUGE_VAL, 1};
  if (p.E > P::kExperts) return best;
  const double experts = p.E < p.rows_max ? p.E : (double)p.rows_max, rows = p.rows_max / experts;
  const double spread = experts > 1 ? sqrt(rows) : 0.0;
  double tiles = 0.0;
  for (int z = -2; z <= 2; ++z) {
    const double some = ceil((rows + z * spread) / P::kTokens);
    tiles += (some > 1 ? some : 1) / 5;
  }
  const int channels = op == kGated ? kBlock : 2 * kBlock;
  tiles *= experts * ((p.N + channels - 1) / channels);
  const int stages = (p.K + kStageK - 1) / kStageK, steps = (p.K + kStepK - 1) / kStepK;
  for (int split = 1; split <= 8 && (split == 1 || stages >= 2 * split); split *= 2) {
    const int room = split == 8 ? num_sms * 3 / 4 : split == 4 ? num_sms * 19 / 20 : num_sms;
    if (split > 1 && tiles * split > room) break;
    const double us = split == 1 ? ceil(tiles / num_sms) * steps * step
                                 : 2 * ((stages + split - 1) / split) * step + 10.0;
    if (us < best.us) best = {us, split};
  }
  return best;
}

Int8Plan expert_int8_plan(ExpertOp op, const ExpertArgs& p, int num_sms) {
  const Choice few = choose<Few>(op, p, num_sms, 0.43), some = choose<Some>(op, p, num_sms, 0.47),
               many = choose<Many>(op, p, num_sms, 0.51);
  if (few.us <= some.us && few.us <= many.us) return {Few::kTokens, few.split};
  return some.us <= many.us ? Int8Plan{Some::kTokens, some.split}
                            : Int8Plan{Many::kTokens, many.split};
}

cudaError_t launch_expert_int8(ExpertOp op, const ExpertArgs& p, const void* a, const void* b,
                               int num_sms, cudaStream_t st) {
  const Int8Plan plan = expert_int8_plan(op, p, num_sms);
  switch (plan.tokens) {
    case Few::kTokens: return launch<Few>(op, p, a, b, plan.split, num_sms, st);
    case Some::kTokens: return launch<Some>(op, p, a, b, plan.split, num_sms, st);
    default: return launch<Many>(op, p, a, b, plan.split, num_sms, st);
  }
}

}  // namespace moe
