// expert_gemm.cu -- the experts' matrix products over the receive segments on
// the 5th-generation tensor cores.
//
// Rows of expert e are the segment [offset[e], offset[e+1]) of a row buffer.
// Five products share one kernel skeleton:
//   kGated  h  = silu(x Wg^T) * (x Wu^T)            A = x,   B = w13 (K-major)
//   kDown   y  = h W2^T                             A = h,   B = w2  (K-major)
//   kDgate  dh = dy W2, then dg = dh u s (1 + g (1 - s)), du = dh g s with
//           s = 1 / (1 + exp(-g))                   A = dy,  B = w2  (N-major)
//   kDx     dx = [dg du] W13                        A = dgu, B = w13 (N-major)
//   kDw     dW = a^T b over the segment's rows      A = a (M-major), B = b (N-major)
//
// One persistent CTA per SM computes 128 x 256 tiles. One thread copies
// operand tiles (128 bytes along the contiguous axis, 128-byte swizzle) with
// TMA into a ring of stages, one thread issues the tcgen05 products into one
// of two 256-column TMEM accumulators, and eight warps read the other one
// back, so a tile's epilogue runs beside the next tile's products.
// With e4m3 operands the products of one 128-channel block are a partial sum
// that the eight warps multiply by the row's and the block's fp32 scales and
// add up in registers: the accumulators then alternate per block.
//
// Segments end anywhere: rows past a segment's end are computed (they belong
// to the next expert) and not stored; in kDw, where rows are the reduction
// axis, the last block's rows past the end are zeroed in shared memory, in
// both operands, before the products read them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "expert_internal.cuh"
#include "expert_ptx.cuh"
#include "internal.cuh"

namespace moe {
namespace {

constexpr int kTileM = 128;
constexpr int kTileN = 256;
constexpr int kThreads = 384;          // copy, product, TMEM, spare; 8 epilogue warps
constexpr int kEpiWarp0 = 4;
constexpr int kStages = 4;
constexpr int kABytes = kTileM * 128;  // a stage holds 128 bytes of K (or 64 k) per row
constexpr int kBBytes = kTileN * 128;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kEpiBytes = 8 * 2048;    // 32 rows x 64 bytes per epilogue warp
constexpr int kGroupM = 8;             // row tiles that share weight tiles in L2

struct Shared {
  uint64_t full[kStages], empty[kStages];
  uint64_t tfull[2], tempty[2], drain;
  uint32_t tmem;
  int abort;
  uint64_t pair[4];                    // the two warps of a lane quarter exchange amax
  float amax[2][2][kTileM];            // [tile parity][half][row]
  int off[MOE_MAX_EXPERTS + 1];
  int pre[MOE_MAX_EXPERTS + 1];        // row tiles before expert e
};

constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kEpiBytes + (int)sizeof(Shared);
static_assert(kSmemBytes <= 227 * 1024, "shared memory of one CTA");

struct Tile {
  int e;
  int row0;     // first row (kDw: first row of the segment)
  int rows;     // rows of the segment from row0 on (kDw: the reduction length)
  int m0;       // kDw: first gradient row
  int n0;       // first output column
  int kb;       // reduction blocks
};

// Tile t of the launch. Row tiles of one expert are taken in groups of
// kGroupM that walk the columns together, so that concurrent CTAs share both
// operands in L2.
template <int OP>
__device__ __forceinline__ bool get_tile(long long t, const ExpertArgs& p, const Shared& s,
                                         int k_elems, Tile& o) {
  if (OP == kDw) {
    const int mt = (p.M + kTileM - 1) / kTileM;
    const int per = mt * p.nt;
    if (t >= (long long)per * p.E) return false;
    o.e = (int)(t / per);
    const int local = (int)(t - (long long)o.e * per);
    o.row0 = s.off[o.e];
    o.rows = s.off[o.e + 1] - o.row0;
    const int g = local / (kGroupM * p.nt), gs = min(kGroupM, mt - g * kGroupM);
    const int idx = local - g * kGroupM * p.nt;
    o.m0 = (g * kGroupM + idx % gs) * kTileM;
    o.n0 = idx / gs;
    o.kb = (o.rows + 63) >> 6;
    return true;
  }
  if (t >= (long long)s.pre[p.E] * p.nt) return false;
  int lo = 0, hi = p.E - 1;  // largest e with pre[e] * nt <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((long long)s.pre[mid] * p.nt <= t) lo = mid;
    else hi = mid - 1;
  }
  o.e = lo;
  const long long local = t - (long long)s.pre[lo] * p.nt;
  const int mt = s.pre[lo + 1] - s.pre[lo];
  const int g = (int)(local / ((long long)kGroupM * p.nt));
  const int gs = min(kGroupM, mt - g * kGroupM);
  const int idx = (int)(local - (long long)g * kGroupM * p.nt);
  const int m = g * kGroupM + idx % gs;
  o.row0 = s.off[lo] + m * kTileM;
  o.rows = s.off[lo + 1] - o.row0;
  o.m0 = 0;
  o.n0 = idx / gs;
  o.kb = (p.K + k_elems - 1) / k_elems;
  return true;
}

// The segments and the row tiles before each expert, once per CTA. Offsets
// are held to [0, rows_max] and to ascending order, so no row index that
// follows from them leaves a row buffer.
__device__ __forceinline__ void load_segments(const ExpertArgs& p, Shared& s) {
  for (int e = threadIdx.x; e <= p.E; e += kThreads) {
    const long long o = p.offset[e];
    s.off[e] = (int)(o < 0 ? 0 : o > p.rows_max ? p.rows_max : o);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0, top = s.off[0];
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int end = e < p.E ? s.off[e + 1] : 0;
      for (int d = 1; d < 32; d <<= 1) {  // running maximum: ascending ends
        const int v = __shfl_up_sync(~0u, end, d);
        if (lane >= d) end = max(end, v);
      }
      end = max(end, top);
      int begin = __shfl_up_sync(~0u, end, 1);
      if (lane == 0) begin = top;
      top = __shfl_sync(~0u, end, 31);
      const int n = e < p.E ? max(end - begin, 0) : 0;
      const int tiles = (n + kTileM - 1) / kTileM;
      int sum = tiles;
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(~0u, sum, d);
        if (lane >= d) sum += v;
      }
      __syncwarp();
      if (e < p.E) {
        s.pre[e] = carry + sum - tiles;
        s.off[e + 1] = max(end, begin);
      }
      carry += __shfl_sync(~0u, sum, 31);
      __syncwarp();
    }
    if (lane == 0) s.pre[p.E] = carry;
  }
  __syncthreads();
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// 1 / (1 + exp(-g)); exp(-g) = +inf gives 0.
__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }
// g / (1 + exp(-g)). __fdividef returns 0 for divisors above 2^126 (there the
// quotient is below every value that a product with it could show).
__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

// ---- row-coalesced access of a warp's 32 x 32 bf16 tile --------------------
// Each lane holds one row; the tile goes through 2 KB of shared memory
// (16-byte units, swizzled by row so that neither side has bank conflicts) so
// that global accesses cover 64-byte row pieces.
__device__ __forceinline__ int unit_at(int row, int u) { return row * 4 + (u ^ ((row >> 1) & 3)); }

__device__ __forceinline__ void tile_put(uint4* buf, int lane, const uint32_t (&v)[16]) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
    buf[unit_at(lane, u)] = make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
}

__device__ __forceinline__ void tile_get(const uint4* buf, int lane, uint32_t (&v)[16]) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint4 q = buf[unit_at(lane, u)];
    v[4 * u] = q.x;
    v[4 * u + 1] = q.y;
    v[4 * u + 2] = q.z;
    v[4 * u + 3] = q.w;
  }
}

// Rows [0, rows) and 16-byte units [0, units) of the tile at `out` (row pitch
// in bytes).
__device__ __forceinline__ void tile_store(const uint4* buf, int lane, uint8_t* out,
                                           long long pitch, int rows, int units) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2), u = lane & 3;
    if (r < rows && u < units) *reinterpret_cast<uint4*>(out + r * pitch + u * 16) = buf[unit_at(r, u)];
  }
}

__device__ __forceinline__ void tile_load(uint4* buf, int lane, const uint8_t* in, long long pitch,
                                          int rows, int units) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2), u = lane & 3;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && u < units) v = *reinterpret_cast<const uint4*>(in + r * pitch + u * 16);
    buf[unit_at(r, u)] = v;
  }
}

// bf16 columns [0, cols) of the lanes' rows to `out` (row pitch in elements);
// cols is a multiple of 8.
__device__ __forceinline__ void put_store(uint4* buf, int lane, const uint32_t (&v)[16],
                                          uint16_t* out, long long pitch, int rows, int cols) {
  tile_put(buf, lane, v);
  __syncwarp();
  tile_store(buf, lane, reinterpret_cast<uint8_t*>(out), 2 * pitch, rows, cols >> 3);
  __syncwarp();
}

__device__ __forceinline__ void load_get(uint4* buf, int lane, uint32_t (&v)[16],
                                         const uint16_t* in, long long pitch, int rows, int cols) {
  tile_load(buf, lane, reinterpret_cast<const uint8_t*>(in), 2 * pitch, rows, cols >> 3);
  __syncwarp();
  tile_get(buf, lane, v);
  __syncwarp();
}

// ---- epilogues of a finished bf16 accumulator ------------------------------
// taddr: the warp's lanes and the accumulator's first column. half: which of
// the two warps that share the lanes (each takes half of the columns).
template <int OP>
__device__ __forceinline__ void epilogue_bf16(const ExpertArgs& p, const Tile& t, uint32_t taddr,
                                              int half, int quarter, int lane, uint4* buf,
                                              bool zero) {
  const int wrow = quarter * 32;
  if constexpr (OP == kGated) {
    const int rows = t.rows - wrow;
    const long long row = (long long)t.row0 + wrow;
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
      const int c = t.n0 * 128 + half * 64 + j * 32;
      uint32_t g[32], u[32], h[16];
      tc_ld32(g, taddr + half * 64 + j * 32);
      tc_ld32(u, taddr + 128 + half * 64 + j * 32);
      tc_wait_ld();
      tc_loaded(g);
      tc_loaded(u);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float g0 = __uint_as_float(g[2 * i]), g1 = __uint_as_float(g[2 * i + 1]);
        const float u0 = __uint_as_float(u[2 * i]), u1 = __uint_as_float(u[2 * i + 1]);
        h[i] = bf16x2(silu(g0) * u0, silu(g1) * u1);
      }
      put_store(buf, lane, h, static_cast<uint16_t*>(p.out) + row * p.F + c, p.F, rows, p.F - c);
      if (p.gu_out) {
        uint16_t* gu = p.gu_out + row * 2 * p.F + c;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          h[i] = bf16x2(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]));
        put_store(buf, lane, h, gu, 2ll * p.F, rows, p.F - c);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          h[i] = bf16x2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
        put_store(buf, lane, h, gu + p.F, 2ll * p.F, rows, p.F - c);
      }
    }
  } else if constexpr (OP == kDgate) {
    const int rows = t.rows - wrow;
    const long long row = (long long)t.row0 + wrow;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      const int c = t.n0 * kTileN + half * 128 + j * 32;
      uint32_t g[16], u[16], d[32];
      const uint16_t* gu = p.gu + row * 2 * p.F + c;
      load_get(buf, lane, g, gu, 2ll * p.F, rows, p.F - c);
      load_get(buf, lane, u, gu + p.F, 2ll * p.F, rows, p.F - c);
      tc_ld32(d, taddr + half * 128 + j * 32);
      tc_wait_ld();
      tc_loaded(d);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float d0 = __uint_as_float(d[2 * i]), d1 = __uint_as_float(d[2 * i + 1]);
        const float g0 = lo_f(g[i]), g1 = hi_f(g[i]), u0 = lo_f(u[i]), u1 = hi_f(u[i]);
        const float s0 = sigmoid(g0), s1 = sigmoid(g1);
        // d silu(g) / dg = s (1 + g (1 - s))
        g[i] = bf16x2(d0 * u0 * s0 * (1.0f + g0 * (1.0f - s0)),
                      d1 * u1 * s1 * (1.0f + g1 * (1.0f - s1)));
        u[i] = bf16x2(d0 * g0 * s0, d1 * g1 * s1);
      }
      uint16_t* out = static_cast<uint16_t*>(p.out) + row * 2 * p.F + c;
      put_store(buf, lane, g, out, 2ll * p.F, rows, p.F - c);
      put_store(buf, lane, u, out + p.F, 2ll * p.F, rows, p.F - c);
    }
  } else {
    const int rows = OP == kDw ? p.M - t.m0 - wrow : t.rows - wrow;
    const long long row = OP == kDw ? (long long)t.e * p.M + t.m0 + wrow : (long long)t.row0 + wrow;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      const int c = t.n0 * kTileN + half * 128 + j * 32;
      uint32_t o[16];
      if (zero) {  // a segment without rows
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = 0u;
      } else {
        uint32_t d[32];
        tc_ld32(d, taddr + half * 128 + j * 32);
        tc_wait_ld();
        tc_loaded(d);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          o[i] = bf16x2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]));
      }
      put_store(buf, lane, o, static_cast<uint16_t*>(p.out) + row * p.N + c, p.N, rows, p.N - c);
    }
  }
}

__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s) {
  const uint64_t v = (uint64_t)lo | ((uint64_t)hi << 32);
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}
__device__ __forceinline__ uint64_t both(float s) {
  const uint32_t u = __float_as_uint(s);
  return (uint64_t)u | ((uint64_t)u << 32);
}
__device__ __forceinline__ float part(const uint64_t (&acc)[64], int i) {
  return __uint_as_float((uint32_t)(acc[i >> 1] >> (32 * (i & 1))));
}

// With e4m3 operands an epilogue thread holds 128 sums. The CTA launches with
// 12 warps x 168 registers a thread; the first four keep 56 and the other
// eight take 224 (4 x 56 + 8 x 224 = 12 x 168).
template <bool FP8>
__device__ __forceinline__ void give_registers() {
  if constexpr (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
}
template <bool FP8>
__device__ __forceinline__ void take_registers() {
  if constexpr (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
}

template <int OP, bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
    k_expert_gemm(const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_b, const ExpertArgs p) {
  constexpr bool kAmn = OP == kDw;
  constexpr bool kBmn = OP == kDw || OP == kDgate || OP == kDx;
  constexpr int kElems = FP8 ? 128 : 64;  // reduction elements of one stage
  constexpr uint32_t kIdesc = mma_desc(FP8, kAmn, kBmn, kTileM, kTileN);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint4* epi = reinterpret_cast<uint4*>(smem + kStages * kStageBytes);
  Shared& s = *reinterpret_cast<Shared*>(smem + kStages * kStageBytes + kEpiBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 2) tc_alloc(smem_u32(&s.tmem), 512);
  if (threadIdx.x == 0) {
    s.abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.tfull[i]), 1);
      mbar_init(smem_u32(&s.tempty[i]), 8);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&s.pair[i]), 2);
    mbar_init(smem_u32(&s.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  pdl_wait();  // the segments and the operands come from earlier kernels
  load_segments(p, s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const WaitCtl ctl{&s.abort, p.wait_limit, p.status};

  if (warp < kEpiWarp0) {
    give_registers<FP8>();
    if (warp == 0) {
      if (lane == 0) {
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        Tile t;
        for (long long ti = blockIdx.x; ok && get_tile<OP>(ti, p, s, kElems, t); ti += gridDim.x) {
          const int a_copies =
              kAmn ? 0 : (min(t.rows, kTileM) + p.a_box - 1) / p.a_box;
          const uint32_t bytes = kAmn ? kStageBytes : a_copies * p.a_box * 128 + kBBytes;
          for (int kb = 0; kb < t.kb; ++kb) {
            if (!mbar_wait(smem_u32(&s.empty[st]), ph ^ 1, ctl)) {
              ok = false;
              break;
            }
            const uint32_t bar = smem_u32(&s.full[st]);
            const uint32_t a = smem_u32(smem + st * kStageBytes), b = a + kABytes;
            mbar_expect(bar, bytes);
            if constexpr (kAmn) {
              for (int i = 0; i < 2; ++i)
                tma_load_2d(a + i * 8192, &map_a, bar, t.m0 + i * 64, t.row0 + kb * 64);
            } else {
              for (int i = 0; i < a_copies; ++i)
                tma_load_2d(a + i * p.a_box * 128, &map_a, bar, kb * kElems, t.row0 + i * p.a_box);
            }
            if constexpr (OP == kDw) {
              for (int i = 0; i < 4; ++i)
                tma_load_2d(b + i * 8192, &map_b, bar, t.n0 * kTileN + i * 64, t.row0 + kb * 64);
            } else if constexpr (kBmn) {
              for (int i = 0; i < 4; ++i)
                tma_load_3d(b + i * 8192, &map_b, bar, t.n0 * kTileN + i * 64, kb * 64, t.e);
            } else if constexpr (OP == kGated) {
              tma_load_3d(b, &map_b, bar, kb * kElems, t.n0 * 128, t.e);
              tma_load_3d(b + 16384, &map_b, bar, kb * kElems, p.F + t.n0 * 128, t.e);
            } else {
              tma_load_3d(b, &map_b, bar, kb * kElems, t.n0 * kTileN, t.e);
              tma_load_3d(b + 16384, &map_b, bar, kb * kElems, t.n0 * kTileN + 128, t.e);
            }
            if (issued < kStages) ++issued;
            if (++st == kStages) {
              st = 0;
              ph ^= 1;
            }
          }
        }
        // copies in flight land before the CTA ends, also when a wait gave up
        for (int i = 0; i < issued; ++i) {
          if (--st < 0) {
            st = kStages - 1;
            ph ^= 1;
          }
          mbar_drain(smem_u32(&s.full[st]), ph);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      int st = 0, as = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      Tile t;
      for (long long ti = blockIdx.x; ok && get_tile<OP>(ti, p, s, kElems, t); ti += gridDim.x) {
        if (t.kb == 0) continue;
        for (int kb = 0; kb < t.kb; ++kb) {
          if (FP8 || kb == 0) {
            ok = mbar_wait(smem_u32(&s.tempty[as]), aph ^ 1, ctl);
            tc_fence_after();
          }
          ok = ok && mbar_wait(smem_u32(&s.full[st]), ph, ctl);
          ok = __all_sync(~0u, ok);
          if (!ok) break;
          const uint32_t a = smem_u32(smem + st * kStageBytes), b = a + kABytes;
          int ksteps = 4;
          if constexpr (OP == kDw) {
            const int valid = t.rows - kb * 64;
            if (valid < 64) {  // rows of the next segment: zero them in both operands
              ksteps = (valid + 15) >> 4;
              uint4* base = reinterpret_cast<uint4*>(smem + st * kStageBytes);
              const int lines = ksteps * 16 - valid;
              for (int i = lane; i < lines * 8 * 6; i += 32) {
                const int chunk = i / (lines * 8), r = i - chunk * lines * 8;
                base[chunk * 512 + valid * 8 + r] = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_async_smem();
              __syncwarp();
            }
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t d = tmem + as * kTileN;
            uint64_t da = kAmn ? smem_desc(a, 8192, 1024) : smem_desc(a, 16, 1024);
            uint64_t db = kBmn ? smem_desc(b, 8192, 1024) : smem_desc(b, 16, 1024);
            for (int k = 0; k < ksteps; ++k) {
              tc_mma<FP8>(d, da, db, kIdesc, (FP8 ? 0 : kb) > 0 || k > 0);
              // 16 k of bf16 (32 of e4m3): 32 bytes along K, or 16 lines of 128 bytes
              da += (kAmn ? 2048 : 32) >> 4;
              db += (kBmn ? 2048 : 32) >> 4;
            }
            tc_commit(smem_u32(&s.empty[st]));
            if (FP8 || kb == t.kb - 1) tc_commit(smem_u32(&s.tfull[as]));
          }
          __syncwarp();
          if (++st == kStages) {
            st = 0;
            ph ^= 1;
          }
          if (FP8 || kb == t.kb - 1) {
            as ^= 1;
            if (as == 0) aph ^= 1;
          }
        }
      }
      if (lane == 0) {  // products in flight end before TMEM is freed
        tc_commit(smem_u32(&s.drain));
        mbar_drain(smem_u32(&s.drain), 0);
      }
      __syncwarp();
    }
  } else {
    take_registers<FP8>();
    const int ew = warp - kEpiWarp0, quarter = warp & 3, half = ew >> 2;
    uint4* buf = epi + ew * 128;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    int as = 0;
    uint32_t aph = 0, parity = 0;
    bool ok = true;
    Tile t;
    for (long long ti = blockIdx.x; ok && get_tile<OP>(ti, p, s, kElems, t); ti += gridDim.x) {
      if constexpr (!FP8) {
        if (t.kb > 0) {
          ok = __all_sync(~0u, mbar_wait(smem_u32(&s.tfull[as]), aph, ctl));
          if (!ok) break;
          tc_fence_after();
        }
        epilogue_bf16<OP>(p, t, tmem + lanes + as * kTileN, half, quarter, lane, buf, t.kb == 0);
        if (t.kb > 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.tempty[as]));
          as ^= 1;
          if (as == 0) aph ^= 1;
        }
      } else {
        // columns of this thread: kGated 64 of gate and the same 64 of up,
        // kDown 128 in a row; two groups of 64, one weight block each
        const int r = quarter * 32 + lane;
        const bool mine = r < t.rows;
        const float* sa = p.sa + ((long long)t.row0 + (mine ? r : 0)) * t.kb;
        const int blocks = OP == kGated ? 2 * p.F >> 7 : p.N >> 7;
        const int b0 = OP == kGated ? t.n0 : t.n0 * 2 + half;
        const int b1 = OP == kGated ? (p.F >> 7) + t.n0 : b0;
        const float* sb0 = p.sb + ((long long)t.e * blocks + min(b0, blocks - 1)) * t.kb;
        const float* sb1 = p.sb + ((long long)t.e * blocks + min(b1, blocks - 1)) * t.kb;
        const uint32_t c0 = OP == kGated ? half * 64 : half * 128;
        const uint32_t c1 = OP == kGated ? 128 + half * 64 : half * 128 + 64;
        uint64_t acc[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = 0ull;
        float a_next = __ldg(sa), b0_next = __ldg(sb0), b1_next = __ldg(sb1);
        for (int kb = 0; kb < t.kb; ++kb) {
          const uint64_t s0 = both(a_next * b0_next), s1 = both(a_next * b1_next);
          if (kb + 1 < t.kb) {
            a_next = __ldg(sa + kb + 1);
            b0_next = __ldg(sb0 + kb + 1);
            b1_next = __ldg(sb1 + kb + 1);
          }
          ok = __all_sync(~0u, mbar_wait(smem_u32(&s.tfull[as]), aph, ctl));
          if (!ok) break;
          tc_fence_after();
          const uint32_t ta = tmem + lanes + as * kTileN;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint32_t v[32];
            tc_ld32(v, ta + (g < 2 ? c0 : c1) + (g & 1) * 32);
            tc_wait_ld();
            tc_loaded(v);
            if (g == 3) {  // all read: the accumulator may be overwritten
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&s.tempty[as]));
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              fma2(acc[g * 16 + i], v[2 * i], v[2 * i + 1], g < 2 ? s0 : s1);
          }
          as ^= 1;
          if (as == 0) aph ^= 1;
        }
        if (!ok) break;
        const int wrow = quarter * 32, rows = t.rows - wrow;
        const long long row = (long long)t.row0 + wrow;
        if constexpr (OP == kDown) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int c = t.n0 * kTileN + half * 128 + g * 32;
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = bf16x2(part(acc, g * 32 + 2 * i), part(acc, g * 32 + 2 * i + 1));
            put_store(buf, lane, o, static_cast<uint16_t*>(p.out) + row * p.N + c, p.N, rows,
                      p.N - c);
          }
        } else {
          // h = silu(g) u, then e4m3 codes with one scale for the tile's 128
          // columns of the row: its largest magnitude comes from this thread
          // and the one of the other half
          float h[64], m = 0.0f;
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            h[i] = silu(part(acc, i)) * part(acc, 64 + i);
            m = fmaxf(m, fabsf(h[i]));
          }
          s.amax[parity][half][r] = m;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.pair[quarter]));
          ok = __all_sync(~0u, mbar_wait(smem_u32(&s.pair[quarter]), parity, ctl));
          if (!ok) break;
          m = fmaxf(m, s.amax[parity][half ^ 1][r]);
          parity ^= 1;  // the other buffer next: this one is read until then
          const float scale = __fdiv_rn(m, 448.0f);
          if (mine && half == 0) p.out_scale[((long long)t.row0 + r) * (p.F >> 7) + t.n0] = scale;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t q[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float* f = h + 16 * u + 4 * w;
              uint32_t codes = 0;
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const float x0 = scale > 0.0f ? __fdiv_rn(f[2 * b], scale) : 0.0f;
                const float x1 = scale > 0.0f ? __fdiv_rn(f[2 * b + 1], scale) : 0.0f;
                codes |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE,
                                                            __NV_E4M3)
                         << (16 * b);
              }
              q[w] = codes;
            }
            buf[unit_at(lane, u)] = make_uint4(q[0], q[1], q[2], q[3]);
          }
          __syncwarp();
          tile_store(buf, lane,
                     static_cast<uint8_t*>(p.out) + row * p.F + t.n0 * 128 + half * 64, p.F, rows, 4);
          __syncwarp();
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tc_dealloc(tmem, 512);
}

// ---- host side -------------------------------------------------------------
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) !=
            cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// A row-major tensor [planes][rows][cols] of bf16 or bytes; copies of
// box_rows rows x 128 bytes, 128-byte swizzle, zeros outside.
cudaError_t make_map(CUtensorMap* m, const void* base, bool fp8, long long cols, long long rows,
                     long long planes, int box_rows) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return cudaErrorNotSupported;
  const long long elt = fp8 ? 1 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)(cols * elt), (cuuint64_t)(cols * elt * rows)};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / elt), (cuuint32_t)box_rows, 1};
  const cuuint32_t ones[3] = {1, 1, 1};
  const CUresult rc =
      enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
          planes > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, ones,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return rc == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int OP, bool FP8>
cudaError_t launch(const ExpertArgs& p, const void* a, const void* b, int num_sms,
                   cudaStream_t st) {
  CUtensorMap ma, mb;
  cudaError_t e;
  if (OP == kDw) {
    e = make_map(&ma, a, false, p.M, p.rows_max, 0, 64);
    if (e == cudaSuccess) e = make_map(&mb, b, false, p.N, p.rows_max, 0, 64);
  } else {
    e = make_map(&ma, a, FP8, p.K, p.rows_max, 0, p.a_box);
    if (e == cudaSuccess) {
      if (OP == kGated) e = make_map(&mb, b, FP8, p.K, 2ll * p.F, p.E, 128);
      else if (OP == kDown) e = make_map(&mb, b, FP8, p.K, p.N, p.E, 128);
      else e = make_map(&mb, b, false, p.N, p.K, p.E, 64);
    }
  }
  if (e != cudaSuccess) return e;
  // Row tiles are at most one per 128 rows plus one per segment.
  const long long segments = p.E < p.rows_max ? p.E : p.rows_max;
  const long long tiles = OP == kDw ? (long long)((p.M + kTileM - 1) / kTileM) * p.nt * p.E
                                    : (p.rows_max / kTileM + segments) * p.nt;
  const int grid = (int)(tiles < num_sms ? tiles : num_sms);
  return launch_pdl(k_expert_gemm<OP, FP8>, dim3(grid), dim3(kThreads), kSmemBytes, st, ma, mb, p);
}

template <int OP, bool FP8>
cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(k_expert_gemm<OP, FP8>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess || !FP8) return e;
  // The register split (4 warps x 56, 8 warps x 224) spends exactly 12 x 168.
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, k_expert_gemm<OP, FP8>);
  if (e != cudaSuccess) return e;
  return attr.numRegs >= 168 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

}  // namespace

cudaError_t expert_gemm_prepare() {
  cudaError_t e = prepare<kGated, false>();
  if (e == cudaSuccess) e = prepare<kGated, true>();
  if (e == cudaSuccess) e = prepare<kDown, false>();
  if (e == cudaSuccess) e = prepare<kDown, true>();
  if (e == cudaSuccess) e = prepare<kDgate, false>();
  if (e == cudaSuccess) e = prepare<kDx, false>();
  if (e == cudaSuccess) e = prepare<kDw, false>();
  return e;
}

cudaError_t launch_expert_gemm(ExpertOp op, bool fp8, const ExpertArgs& args, const void* a,
                               const void* b, int num_sms, cudaStream_t st) {
  ExpertArgs p = args;
  p.a_box = 128;
  p.nt = op == kGated ? (p.F + 127) / 128 : (p.N + kTileN - 1) / kTileN;
  switch (op) {
    case kGated:
      return fp8 ? launch<kGated, true>(p, a, b, num_sms, st)
                 : launch<kGated, false>(p, a, b, num_sms, st);
    case kDown:
      return fp8 ? launch<kDown, true>(p, a, b, num_sms, st)
                 : launch<kDown, false>(p, a, b, num_sms, st);
    case kDgate: return launch<kDgate, false>(p, a, b, num_sms, st);
    case kDx: return launch<kDx, false>(p, a, b, num_sms, st);
    default: return launch<kDw, false>(p, a, b, num_sms, st);
  }
}

}  // namespace moe
