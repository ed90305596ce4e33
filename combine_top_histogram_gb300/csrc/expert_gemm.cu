// expert_gemm.cu -- the experts' matrix products over the receive segments on
// the 5th-generation tensor cores.
//
// Rows of expert e are the segment [offset[e], offset[e+1]) of a row buffer.
// Five products share one kernel skeleton:
//   kGated  h  = silu(x Wg^T) * (x Wu^T)            A = x,   B = w13 (K-major)
//   kDown   y  = h W2^T                             A = h,   B = w2  (K-major)
//   kDgate  dh = dy W2, then dg = dh u s (1 + g (1 - s)), du = dh g s with
//           s = 1 / (1 + exp(-g))                   A = dy,  B = w2  (N-major)
//           (dg and du rounded to bf16, which kDx and kDw feed to the tensor
//           cores: the gradients' relative error against 64 bits is then 0.0024,
//           with rounded results alone 0.0017; held in two bf16 parts each,
//           they would double those products)
//   kDx     dx = [dg du] W13                        A = dgu, B = w13 (N-major)
//   kDw     dW = a^T b over the segment's rows      A = a (M-major), B = b (N-major)
//
// One persistent CTA per SM. A CTA computes 128 x 256 tiles, or the two CTAs
// of a cluster compute 256 x 256 tiles together (CG = 2): each holds its 128
// rows of A and accumulator and half of B's columns, and the first CTA issues
// the products of both. One warp per CTA copies operand tiles (128 bytes
// along the contiguous axis, 128-byte swizzle) with TMA into a ring of stages,
// one warp issues the tcgen05 products into one of two 256-column TMEM
// accumulators, and eight warps read the other one back, so a tile's epilogue
// runs beside the next tile's products. Where tiles are few they are 128
// columns wide. The copy and issue warps run converged, one elected lane
// executing: as a branch of one lane they kept addresses and descriptors in
// vector registers and bound the products (gated bf16, E = 8, 65536 rows by
// Zipf(1.2), H = 4096, F = 1408: 903 us, against 791).
// With e4m3 operands the products of one 128-channel block are a partial sum
// that the eight warps multiply by the row's and the block's fp32 scales and
// add up in registers: the accumulators then alternate per block.
//
// What bounds it: of bf16 with many rows the tensor pipe (pairs: 94 % of the
// SMs' active cycles in kGated and kDx, 81 % in kDw; 1.91 PFLOP/s in that case,
// 1.66 where passes follow each other for long and the card is at its power
// cap), without pairs shared memory, whose 128 bytes a cycle serve the copies
// and the products (96 KB for a block's 512 cycles). Of e4m3 with many rows
// the way of the accumulators, two of which fill the tensor memory, between
// the products and the warps that scale them (820 cycles a block, 512 of
// products; E = 64, 32768 rows, H = 7168, F = 2048: 2.15 PFLOP/s, 1.96 for
// long). With few rows per expert HBM (E = 256, 8192 rows: 0.99 of the copy
// rate).
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
#include "expert_math.cuh"
#include "expert_ptx.cuh"
#include "internal.cuh"

namespace moe {
namespace {

constexpr int kTileM = 128;            // rows of one CTA's accumulator
constexpr int kAccColumns = 256;       // tensor-memory columns of one accumulator
constexpr int kThreads = 384;          // copy, product, TMEM, spare; 8 epilogue warps
constexpr int kEpiWarp0 = 4;
constexpr int kABytes = kTileM * 128;  // a stage holds 128 bytes of K (or 64 k) per row
// Shared memory of a kernel: the ring of stages, and what the epilogue warps
// pass their results through: 32 rows x 64 bytes per warp, or (kOut) the
// warp's whole 32 x TN / 2 bf16 results, which the copy engine then writes
// beside the next tile's products; those take the room of one stage.
template <int OP, bool FP8, int CG, int TN>
struct Plan {
  static constexpr int kBRows = TN / CG;  // rows (or columns) of B in one CTA
  static constexpr int kStageBytes = kABytes + kBRows * 128;
  static constexpr bool kOut = (OP == kDown && FP8) || (OP == kDw && TN == 128);
  static constexpr int kStages = (kStageBytes > 32768 ? 4 : 6) - (kOut ? CG : 0);
  static constexpr int kWarpBytes = kOut ? TN / 128 * 4096 : 2048;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kEpiBytes = 8 * kWarpBytes;
};
constexpr int kMaxStages = 6;
constexpr int kGroupM = 8;             // row tiles that share weight tiles in L2

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2], drain;
  uint64_t tail[kMaxStages];           // kDw, second CTA: its copies of a segment's last block
  uint32_t tmem;
  int abort, uneven;
  uint32_t announced;                  // pairs: stages whose copies this CTA has announced,
  uint32_t tails, tail_phase;          // in kDw's second CTA: the stages whose last ones were
  uint32_t tails_sent, tails_done;     // for `tail`, these barriers' parities, how many there
                                       // were and how many its other warp has handed on
  uint64_t pair[4];                    // the two warps of a lane quarter exchange amax
  float amax[2][2][kTileM];            // [tile parity][half][row]
  uint64_t sempty[2];                  // the epilogue has read scale[i]
  float2 scale[2][kTileM];             // FP8: row scale x scales of the tile's two weight blocks
  int off[MOE_MAX_EXPERTS + 1];
  int pre[MOE_MAX_EXPERTS + 1];        // row tiles before expert e (kDw: see sort_segments)
};

template <int OP, bool FP8, int CG, int TN>
constexpr int smem_bytes() {
  using P = Plan<OP, FP8, CG, TN>;
  constexpr int bytes = 1024 + P::kRingBytes + P::kEpiBytes + (int)sizeof(Shared);
  static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
  // more than half of an SM's: a second CTA, and with it a second allocation
  // of the tensor memory, never shares it
  static_assert(bytes > 114 * 1024, "one CTA per SM");
  return bytes;
}

struct Tile {
  int e;
  int row0;     // this CTA's first row (kDw: first row of the segment)
  int rows;     // rows of the segment from row0 on (kDw: the reduction length)
  int m0;       // kDw: this CTA's first gradient row
  int n0;       // column tile
  int kb;       // reduction blocks
};

// The tiles of one CTA (or pair), in order: tile0, tile0 + step, ... of the
// launch. Row tiles of one expert are taken in groups of kGroupM that walk the
// columns together, so that concurrent CTAs share both operands in L2. Each
// role walks for itself; a step costs two divisions and, within an expert or
// to one of the next few, no search.
// kDw's tiles take as long as their expert has rows. Where some have many more
// than others, the experts come by falling rows (sort_segments) and every
// second step goes backwards over the CTAs, so that those with the long tiles
// of one step get the short ones of the next (Zipf(1.2) over 8 experts, 76
// pairs: the last pair ends 7 and 6 % after the mean for dW2 and dW13 of the
// skewed training layer, without 17 and 8 %; its backward pass 2640 / 2570 us).
// Even ones keep the plain order, which costs less to walk (E = 64 of 256 rows
// each: 464 / 480 us).
template <int OP, int CG>
struct Walk {
  static constexpr int kRows = kTileM * CG;
  const ExpertArgs& p;
  const Shared& s;
  const int k_elems, rank, first, step, mt_w;
  int t, e, base, per;  // tile, its expert, the expert's first tile and tiles
  int place = 0;        // kDw: the expert's place by falling rows
  bool uneven, back = true;  // kDw: some experts' rows are many more; this step goes backwards

  __device__ __forceinline__ Walk(const ExpertArgs& pa, const Shared& sh, int ke, int rk, int tile0,
                                  int st)
      : p(pa), s(sh), k_elems(ke), rank(rk), first(tile0), step(st),
        mt_w(OP == kDw ? (pa.M + kRows - 1) / kRows : 0), t(tile0 - st), e(0), base(0) {
    per = tiles(0);
    uneven = OP == kDw && sh.uneven;
    if (uneven) e = sh.pre[0];
  }

  __device__ __forceinline__ int tiles(int x) const {
    return (OP == kDw ? mt_w : s.pre[x + 1] - s.pre[x]) * p.nt;
  }

  __device__ __forceinline__ bool next(Tile& o) {
    t += step;
    uint32_t local;  // tile of the expert
    if (OP == kDw) {
      int at = t;
      if (uneven) {
        back = !back;
        if (back) at += step - 1 - 2 * first;
      }
      if (at >= mt_w * p.E * p.nt) return false;
      if (at < base || at - base >= per) {
        place = at / per;
        base = place * per;
        e = uneven ? s.pre[place] : place;
      }
      local = at - base;
    } else {
      if (t >= s.pre[p.E] * p.nt) return false;
      for (int i = 0; i < 4 && t - base >= per; ++i) {
        base += per;
        per = tiles(++e);
      }
      if (t - base >= per) {
        int lo = e, hi = p.E - 1;  // largest e with pre[e] * nt <= t
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s.pre[mid] * p.nt <= t) lo = mid;
          else hi = mid - 1;
        }
        e = lo;
        base = s.pre[e] * p.nt;
        per = tiles(e);
      }
      local = t - base;
    }
    const int mt = OP == kDw ? mt_w : s.pre[e + 1] - s.pre[e];
    const uint32_t group = kGroupM * p.nt;
    const uint32_t g = local / group, idx = local - g * group;
    const uint32_t gs = min(kGroupM, mt - (int)g * kGroupM);
    const uint32_t n = gs == kGroupM ? idx / kGroupM : idx / gs;
    const int m = (int)(g * kGroupM + idx - n * gs) * kRows + rank * kTileM;
    o.e = e;
    o.n0 = (int)n;
    if (OP == kDw) {
      o.row0 = s.off[e];
      o.rows = s.off[e + 1] - o.row0;
      o.m0 = m;
      o.kb = (o.rows + 63) >> 6;
    } else {
      o.row0 = s.off[e] + m;
      o.rows = s.off[e + 1] - o.row0;
      o.m0 = 0;
      o.kb = (p.K + k_elems - 1) / k_elems;
    }
    return true;
  }
};

// The segments and the row tiles before each expert, once per CTA. Offsets
// are held to [0, rows_max] and to ascending order, so no row index that
// follows from them leaves a row buffer.
template <int CG>
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
      const int tiles = (n + kTileM * CG - 1) / (kTileM * CG);
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

// kDw: whether some expert has more than 1.5 times the mean of the rows, among
// up to 256 experts (of more, one expert's tiles weigh little) of more than two
// blocks each on average; then the experts by falling rows, equal ones by their
// number, in pre.
__device__ __forceinline__ void sort_segments(const ExpertArgs& p, Shared& s) {
  const long long total = s.off[p.E] - s.off[0];
  int most = 0;
  for (int e = threadIdx.x; e < p.E; e += kThreads) most = max(most, s.off[e + 1] - s.off[e]);
  const bool uneven = __syncthreads_or(p.E <= 256 && total > 128ll * p.E &&
                                       2ll * most * p.E > 3 * total);
  if (threadIdx.x == 0) s.uneven = uneven;
  if (!uneven) return;
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    const int n = s.off[e + 1] - s.off[e];
    int place = 0;
    for (int i = 0; i < p.E; ++i) {
      const int m = s.off[i + 1] - s.off[i];
      place += m > n || (m == n && i < e);
    }
    s.pre[place] = e;
  }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}

// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 32 bytes to memory that is 16-byte aligned at least.
__device__ __forceinline__ void store32(void* to, const uint32_t (&v)[8]) {
  if ((reinterpret_cast<uintptr_t>(to) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    uint4* q = static_cast<uint4*>(to);
    q[0] = make_uint4(v[0], v[1], v[2], v[3]);
    q[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

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
    if (r < rows && u < units)
      *reinterpret_cast<uint4*>(out + r * pitch + u * 16) = buf[unit_at(r, u)];
  }
}

// The 32 x 32 bf16 tile at `in` (row pitch in elements), as tile_store's lanes
// hold it; zeros outside its rows and columns.
__device__ __forceinline__ void tile_fetch(uint4 (&v)[4], int lane, const uint16_t* in,
                                           long long pitch, int rows, int cols) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2), u = lane & 3;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows && u * 8 < cols) v[i] = *reinterpret_cast<const uint4*>(in + r * pitch + u * 8);
  }
}

// A fetched tile, handed to the lanes by row.
__device__ __forceinline__ void tile_turn(uint4* buf, int lane, const uint4 (&in)[4],
                                          uint32_t (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) buf[unit_at(i * 8 + (lane >> 2), lane & 3)] = in[i];
  __syncwarp();
  tile_get(buf, lane, v);
  __syncwarp();
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

// The warp's bf16 results on their way to the copy engine: pieces of 32 rows x
// 64 columns, 128 bytes a row, swizzled as the copies expect. out_begin waits
// until the last copies have read them.
__device__ __forceinline__ int out_unit(int row, int u) {
  return (u >> 3) * 256 + row * 8 + ((u & 7) ^ (row & 7));
}
__device__ __forceinline__ void out_begin(int lane) {
  if (lane == 0) bulk_wait_read();
  __syncwarp();
}

// kDgate: the pre-activations that belong to the 32 columns j of a warp's part
// of the tile, gate and up.
struct GateUp {
  uint4 g[4], u[4];
};
template <int TN>
__device__ __forceinline__ void gate_fetch(GateUp& v, const ExpertArgs& p, const Tile& t, int half,
                                           int quarter, int lane, int j) {
  const int c = t.n0 * TN + half * (TN / 2) + j * 32, rows = t.rows - quarter * 32;
  const uint16_t* gu = p.gu + ((long long)t.row0 + quarter * 32) * 2 * p.F + c;
  tile_fetch(v.g, lane, gu, 2ll * p.F, rows, p.F - c);
  tile_fetch(v.u, lane, gu + p.F, 2ll * p.F, rows, p.F - c);
}

// ---- epilogues of a finished bf16 accumulator ------------------------------
// taddr: the warp's lanes and the accumulator's first column. half: which of
// the two warps that share the lanes (each takes half of the columns).
template <int OP, int TN>
__device__ __forceinline__ void epilogue_bf16(const ExpertArgs& p, const Tile& t, uint32_t taddr,
                                              int half, int quarter, int lane, uint4* buf,
                                              bool zero, GateUp& pre, const CUtensorMap& map_c) {
  const int wrow = quarter * 32;
  if constexpr (OP == kGated) {
    const int rows = t.rows - wrow;
    const long long row = (long long)t.row0 + wrow;
#pragma unroll 1
    for (int j = 0; j < TN / 128; ++j) {
      const int at = half * (TN / 4) + j * 32, c = t.n0 * (TN / 2) + at;
      uint32_t g[32], u[32], h[16];
      tc_ld32(g, taddr + at);
      tc_ld32(u, taddr + TN / 2 + at);
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
    for (int j = 0; j < TN / 64; ++j) {
      const int at = half * (TN / 2) + j * 32, c = t.n0 * TN + at;
      uint32_t g[16], u[16], d[32];
      tile_turn(buf, lane, pre.g, g);
      tile_turn(buf, lane, pre.u, u);
      if (j < TN / 64 - 1)  // beside this part's work
        gate_fetch<TN>(pre, p, t, half, quarter, lane, j + 1);
      tc_ld32(d, taddr + at);
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
  } else if constexpr (OP == kDw && TN == 128) {
    // to the copy engine, which leaves out what lies past the gradient's rows
    // or columns
    const int col = t.n0 * TN + half * 64, row = t.m0 + wrow;
    if (row >= p.M || col >= p.N) return;
    out_begin(lane);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t d[32];
      if (zero) {  // a segment without rows
#pragma unroll
        for (int i = 0; i < 32; ++i) d[i] = 0u;
      } else {
        tc_ld32(d, taddr + half * 64 + j * 32);
        tc_wait_ld();
        tc_loaded(d);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = bf16x2(__uint_as_float(d[8 * u + 2 * i]), __uint_as_float(d[8 * u + 2 * i + 1]));
        buf[out_unit(lane, j * 4 + u)] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(&map_c, smem_u32(buf), col, row, t.e);
      bulk_commit();
    }
  } else {
    const int rows = OP == kDw ? p.M - t.m0 - wrow : t.rows - wrow;
    const long long row = OP == kDw ? (long long)t.e * p.M + t.m0 + wrow : (long long)t.row0 + wrow;
    if (zero) {  // kDw: a segment without rows; half a row of the tile per 16 lanes
      const int c = t.n0 * TN + half * (TN / 2) + (lane & 15) * 8;
      uint16_t* out = static_cast<uint16_t*>(p.out) + (row + (lane >> 4)) * p.N + c;
      if (c < p.N)
        for (int r = lane >> 4; r < min(rows, 32); r += 2, out += 2ll * p.N)
          *reinterpret_cast<uint4*>(out) = make_uint4(0u, 0u, 0u, 0u);
      return;
    }
#pragma unroll 1
    for (int j = 0; j < TN / 64; ++j) {
      const int at = half * (TN / 2) + j * 32, c = t.n0 * TN + at;
      uint32_t d[32], o[16];
      tc_ld32(d, taddr + at);
      tc_wait_ld();
      tc_loaded(d);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        o[i] = bf16x2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]));
      put_store(buf, lane, o, static_cast<uint16_t*>(p.out) + row * p.N + c, p.N, rows, p.N - c);
    }
  }
}

// An epilogue warp has read accumulator `as`: tells the CTA that issues the
// products.
template <int CG>
__device__ __forceinline__ void release(Shared& s, int as) {
  if constexpr (CG == 2) mbar_arrive_relaxed(cluster_addr(smem_u32(&s.tempty[as]), 0));
  else mbar_arrive(smem_u32(&s.tempty[as]));
}

// Rows from `valid` to the next multiple of 16 of a stage's CHUNKS M- or
// N-major operand pieces (64 lines of 128 bytes each) become zero, for the
// tensor cores to read. Whole warp.
template <int CHUNKS>
__device__ __forceinline__ void clear_rows(uint8_t* stage, int valid, int lane) {
  uint4* base = reinterpret_cast<uint4*>(stage);
  const int units = (((valid + 15) & ~15) - valid) * 8;  // 16-byte units of one piece
  for (int i = lane; i < units * CHUNKS; i += 32) {
    const int chunk = i / units, r = i - chunk * units;
    base[chunk * 512 + valid * 8 + r] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_async_smem();
  __syncwarp();
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

// The warp that issues the products: its place in the ring of stages and in
// the two accumulators.
template <class PLAN, int CG, int TN, bool FP8, bool AMN, bool BMN>
struct Issuer {
  static constexpr int kStages = PLAN::kStages, kStageBytes = PLAN::kStageBytes;
  static constexpr uint32_t kIdesc = mma_desc(FP8, AMN, BMN, kTileM * CG, TN);
  // 16 k of bf16 (32 of e4m3): 32 bytes along K, or 16 lines of 128 bytes
  static constexpr uint64_t kA = (AMN ? 2048 : 32) >> 4, kB = (BMN ? 2048 : 32) >> 4;
  const uint32_t full0, empty0, tfull0, tempty0, tmem;
  const uint64_t da0, db0;
  const WaitCtl& ctl;
  int st = 0, as = 0;
  uint32_t ph = 0, aph = 1;

  __device__ __forceinline__ Issuer(Shared& s, uint8_t* smem, uint32_t tm, const WaitCtl& c)
      : full0(smem_u32(s.full)), empty0(smem_u32(s.empty)), tfull0(smem_u32(s.tfull)),
        tempty0(smem_u32(s.tempty)), tmem(tm),
        da0(smem_desc(smem_u32(smem), AMN ? 8192 : 16, 1024)),
        db0(smem_desc(smem_u32(smem) + kABytes, BMN ? 8192 : 16, 1024)), ctl(c) {}

  // Waits for a stage's operands and, where a sum begins, for its accumulator.
  __device__ __forceinline__ bool wait(bool begins) {
    bool ok = mbar_wait<CG == 2>(full0 + st * 8, ph, ctl);
    if (begins) ok = ok && mbar_wait<CG == 2>(tempty0 + as * 8, aph, ctl);
    ok = __all_sync(~0u, ok);
    tc_fence_after();
    return ok;
  }

  // The products of the stage, `steps` of 16 k (e4m3: 32); begins, ends: of
  // the sum in the accumulator.
  __device__ __forceinline__ void block(bool begins, bool ends, int steps) {
    const uint32_t d = tmem + as * kAccColumns;
    const uint64_t da = da0 + (uint64_t)(st * (kStageBytes >> 4));
    const uint64_t db = db0 + (uint64_t)(st * (kStageBytes >> 4));
    if (steps == 4) {
      tc_mma<CG, FP8, 2>(d, da, db, kA, kB, kIdesc, !begins);
      tc_mma<CG, FP8, 2>(d, da + 2 * kA, db + 2 * kB, kA, kB, kIdesc, true);
    } else {
      for (int k = 0; k < steps; ++k)
        tc_mma<CG, FP8, 1>(d, da + k * kA, db + k * kB, 0, 0, kIdesc, !begins || k > 0);
    }
    if (ends) {
      tc_commit<CG>(tfull0 + as * 8);
      as ^= 1;
      if (as == 0) aph ^= 1;
    }
    tc_commit<CG>(empty0 + st * 8);
    if (++st == kStages) {
      st = 0;
      ph ^= 1;
    }
  }
};

// Waits until the last stages that were announced, of `announced` in all, have
// their copies.
template <int STAGES>
__device__ __forceinline__ void drain_stages(Shared& s, uint32_t announced) {
  const uint32_t n = announced < STAGES ? announced : STAGES;
  for (uint32_t i = announced - n; i != announced; ++i)
    mbar_drain(smem_u32(&s.full[i % STAGES]), (i / STAGES) & 1);
}

// After a wait gave up in a pair and both CTAs' warps have left their loops: a
// stage that only one CTA has announced, or whose last block the second CTA
// has not handed on, never completes by itself. The first warps make the
// missing arrivals and wait for what is in flight into either CTA. (No CTA is
// more than the ring's stages ahead: a stage is announced again only after its
// products, and those wait for both.)
template <int OP, int STAGES>
__device__ __forceinline__ void settle_pair(Shared& s, int rank) {
  if (rank == 1) {
    if (OP == kDw) {
      uint32_t left = s.tails_sent - s.tails_done;
      for (uint32_t i = s.announced; left != 0 && i != 0; --i) {
        const uint32_t st = (i - 1) % STAGES;
        if (!((s.tails >> st) & 1)) continue;
        mbar_drain(smem_u32(&s.tail[st]), ((s.tail_phase >> st) & 1) ^ 1);
        if ((threadIdx.x & 31) == 0)
          mbar_arrive_release(cluster_addr(smem_u32(&s.full[st]), 0));
        --left;
      }
    }
  } else {
    uint32_t other;
    asm volatile("ld.shared::cluster.u32 %0, [%1];"
                 : "=r"(other)
                 : "r"(cluster_addr(smem_u32(&s.announced), 1))
                 : "memory");
    const uint32_t most = max(s.announced, other);
    if ((threadIdx.x & 31) == 0)
      for (uint32_t i = min(s.announced, other); i != most; ++i)
        mbar_arrive(smem_u32(&s.full[i % STAGES]));
    __syncwarp();
    drain_stages<STAGES>(s, most);
  }
  __syncwarp();
}

// FP8: two warps keep the scales of the next accumulators ready, so that the
// epilogue warps never wait for memory: for each reduction block the 128 rows'
// scale times those of the tile's two weight blocks. Thread j of 64 serves
// rows j and j + 64 and loads two blocks ahead (four spilled registers that
// the issuing warp of the same register share then missed: 2 % slower).
template <int OP, int CG>
__device__ __forceinline__ void scale_warp(const ExpertArgs& p, Shared& s, const WaitCtl& ctl,
                                           Walk<OP, CG>& walk, int j) {
  constexpr int kAhead = 2;
  int as = 0;
  uint32_t ph = 1;
  Tile t;
  while (walk.next(t)) {
    // a row past the segment's end takes the scales of the segment's first
    const float* a0 = p.sa + (long long)(j < t.rows ? t.row0 + j : s.off[t.e]) * t.kb;
    const float* a1 = p.sa + (long long)(j + 64 < t.rows ? t.row0 + j + 64 : s.off[t.e]) * t.kb;
    const int blocks = OP == kGated ? 2 * p.F >> 7 : p.N >> 7;
    const int n0 = OP == kGated ? t.n0 : 2 * t.n0;
    const int n1 = OP == kGated ? (p.F >> 7) + t.n0 : min(2 * t.n0 + 1, blocks - 1);
    const float* b0 = p.sb + ((long long)t.e * blocks + n0) * t.kb;
    const float* b1 = p.sb + ((long long)t.e * blocks + n1) * t.kb;
    float next[4][kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = min(i, t.kb - 1);
      next[0][i] = __ldg(a0 + k);
      next[1][i] = __ldg(a1 + k);
      next[2][i] = __ldg(b0 + k);
      next[3][i] = __ldg(b1 + k);
    }
    for (int kb = 0; kb < t.kb; kb += kAhead) {
      float now[4][kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int k = min(kb + kAhead + i, t.kb - 1);
#pragma unroll
        for (int q = 0; q < 4; ++q) now[q][i] = next[q][i];
        next[0][i] = __ldg(a0 + k);
        next[1][i] = __ldg(a1 + k);
        next[2][i] = __ldg(b0 + k);
        next[3][i] = __ldg(b1 + k);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (kb + i >= t.kb) break;
        if (!__all_sync(~0u, mbar_wait<CG == 2>(smem_u32(&s.sempty[as]), ph, ctl))) return;
        s.scale[as][j] = make_float2(now[0][i] * now[2][i], now[0][i] * now[3][i]);
        s.scale[as][j + 64] = make_float2(now[1][i] * now[2][i], now[1][i] * now[3][i]);
        __syncwarp();
        if ((j & 31) == 0) mbar_arrive(smem_u32(&s.tfull[as]));
        as ^= 1;
        if (as == 0) ph ^= 1;
      }
    }
  }
}

// Two sums at a time (one issue slot for two fused multiply-adds).
__device__ __forceinline__ void fma2(float2& acc, uint32_t lo, uint32_t hi, float s) {
  acc = __ffma2_rn(make_float2(__uint_as_float(lo), __uint_as_float(hi)), make_float2(s, s), acc);
}

// -a / s rounded to nearest for two values, y = RN(1 / s): the product by the
// reciprocal is within 1.5 units in its last place, and each of two steps adds
// the residual times y (P. Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990: the first
// makes the quotient faithful, the second rounds it correctly). For s between
// 2^-64 and 2^64 only quotients below 2^-40 can differ, whose e4m3 code is a
// signed zero. Of the negative, because a zero then keeps its sign: a = -0
// gives +0, and a = +0 gives -0.
__device__ __forceinline__ float2 minus_quotient(float2 a, float s, float y) {
  const float2 ss = make_float2(s, s), ny = make_float2(-y, -y);
  float2 q = __fmul2_rn(a, ny);
#pragma unroll
  for (int i = 0; i < 2; ++i) q = __ffma2_rn(__ffma2_rn(ss, q, a), ny, q);
  return q;
}

template <int OP, bool FP8, int CG, int TN>
__global__ void __launch_bounds__(kThreads, 1)
    k_expert_gemm(const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_c, const ExpertArgs p) {
  constexpr bool kAmn = OP == kDw;
  constexpr bool kBmn = OP == kDw || OP == kDgate || OP == kDx;
  constexpr int kElems = FP8 ? 128 : 64;  // reduction elements of one stage
  using P = Plan<OP, FP8, CG, TN>;
  static_assert(TN == 256 || (TN == 128 && !FP8 && CG == 1), "tile");
  constexpr int kStages = P::kStages, kStageBytes = P::kStageBytes;
  constexpr bool kPair = CG == 2;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint4* epi = reinterpret_cast<uint4*>(smem + P::kRingBytes);
  Shared& s = *reinterpret_cast<Shared*>(smem + P::kRingBytes + P::kEpiBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kPair ? (int)(blockIdx.x & 1) : 0;  // clusters are pairs of neighbours

  if (warp == 2) tc_alloc<CG>(smem_u32(&s.tmem), 512);
  if (threadIdx.x == 0) {
    s.abort = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), CG);
      mbar_init(smem_u32(&s.empty[i]), 1);
      mbar_init(smem_u32(&s.tail[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.tfull[i]), FP8 ? 3 : 1);  // the products, and two scale warps
      mbar_init(smem_u32(&s.sempty[i]), 8);
      mbar_init(smem_u32(&s.tempty[i]), 8 * CG);
    }
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&s.pair[i]), 2);
    mbar_init(smem_u32(&s.drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
    if constexpr (P::kOut) tma_prefetch_map(&map_c);
  }
  pdl_wait();  // the segments and the operands come from earlier kernels
  load_segments<CG>(p, s);
  if constexpr (OP == kDw) sort_segments(p, s);
  tc_fence_before();
  if constexpr (kPair) cluster_sync();  // both CTAs' barriers exist
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const WaitCtl ctl{&s.abort, kPair ? cluster_addr(smem_u32(&s.abort), rank ^ 1) : 0u, p.wait_limit,
                    p.status};
  Walk<OP, CG> walk(p, s, kElems, rank, blockIdx.x / CG, gridDim.x / CG);

  if (warp < kEpiWarp0) {
    give_registers<FP8>();
    if (warp == 0) {
      int st = 0;
      uint32_t ph = 0, announced = 0, tails = 0, tail_phase = 0, tails_sent = 0;
      bool ok = true;
      Tile t;
      const uint32_t ring = smem_u32(smem);
      const uint32_t full0 = smem_u32(s.full), empty0 = smem_u32(s.empty);
      const uint32_t full0_first = kPair ? cluster_addr(full0, 0) : full0;
      while (ok && walk.next(t)) {
        // uniform, and known to be
        const int blocks = __shfl_sync(~0u, t.kb, 0), e = __shfl_sync(~0u, t.e, 0);
        const int row0 = __shfl_sync(~0u, t.row0, 0), rows = __shfl_sync(~0u, t.rows, 0);
        const int m0 = __shfl_sync(~0u, t.m0, 0), n0 = __shfl_sync(~0u, t.n0, 0);
        // copies cover at least the tile's rows (a pair's always 128)
        const int a_copies = kAmn ? 0 : kPair ? 1 : (min(rows, kTileM) + p.a_box - 1) / p.a_box;
        const uint32_t bytes =
            kAmn || kPair ? kStageBytes : a_copies * p.a_box * 128 + TN * 128;
        for (int kb = 0; kb < blocks; ++kb) {
          ok = __all_sync(~0u, mbar_wait<kPair>(empty0 + st * 8, ph ^ 1, ctl));
          if (!ok) break;
          // a pair's copies all arrive at the first CTA's barrier, except
          // those of a block that the second CTA has to clear rows of first
          uint32_t bar = full0_first + st * 8;
          const uint32_t a = ring + st * kStageBytes, b = a + kABytes;
          if (kPair && OP == kDw && rank == 1 && rows - kb * 64 < 64) {
            bar = smem_u32(&s.tail[st]);
            mbar_expect_elected(bar, bytes);
            bar = cluster_addr(bar, 1);
            tails |= 1u << st;
            tail_phase ^= 1u << st;
            ++tails_sent;
          } else if constexpr (kPair) {
            mbar_expect_relaxed_elected(bar, bytes);
            if (OP == kDw) tails &= ~(1u << st);
          } else {
            mbar_expect_elected(bar, bytes);
          }
          if constexpr (kAmn) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              tma_load_2d<CG>(a + i * 8192, &map_a, bar, m0 + i * 64, row0 + kb * 64);
          } else if constexpr (kPair) {
            tma_load_2d<CG>(a, &map_a, bar, kb * kElems, row0);
          } else {
            for (int i = 0; i < a_copies; ++i)
              tma_load_2d<CG>(a + i * p.a_box * 128, &map_a, bar, kb * kElems, row0 + i * p.a_box);
          }
          // B: the tile's columns, or this CTA's half of them
          if constexpr (kBmn) {
#pragma unroll
            for (int i = 0; i < TN / 64 / CG; ++i) {
              const int n = n0 * TN + rank * 128 + i * 64;
              if constexpr (OP == kDw)
                tma_load_2d<CG>(b + i * 8192, &map_b, bar, n, row0 + kb * 64);
              else
                tma_load_3d<CG>(b + i * 8192, &map_b, bar, n, kb * 64, e);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2 / CG; ++i) {
              const int half = i + rank;  // kGated: gate columns, then up columns
              const int n = OP == kGated ? half * p.F + n0 * (TN / 2) : n0 * TN + half * (TN / 2);
              tma_load_3d<CG>(b + i * (TN / 2 * 128), &map_b, bar, kb * kElems, n, e);
            }
          }
          ++announced;
          if (++st == kStages) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      // Copies in flight land before the CTA (the pair) ends, also when a wait
      // gave up: then a pair may have announced unlike numbers of stages, and
      // settles that below.
      if (kPair && lane == 0) {
        s.announced = announced;
        s.tails = tails;
        s.tail_phase = tail_phase;
        s.tails_sent = tails_sent;
      }
      if (rank == 0 && !(kPair && *ctl.abort)) drain_stages<kStages>(s, announced);
      __syncwarp();
    } else if (kPair && warp == 1 && rank == 1) {
      // The second CTA issues no products. In kDw it clears its rows past a
      // segment's end and then arrives at the first CTA's barrier.
      if constexpr (OP == kDw) {
        int st = 0;
        uint32_t phases = 0;  // bit i: parity of tail[i]'s next phase
        uint32_t handed_on = 0;
        bool ok = true;
        Tile t;
        while (ok && walk.next(t)) {
          st = (st + t.kb) % kStages;
          const int valid = t.rows & 63;
          if (valid == 0) continue;
          const int last = st == 0 ? kStages - 1 : st - 1;
          ok = __all_sync(~0u,
                          mbar_wait<kPair>(smem_u32(&s.tail[last]), (phases >> last) & 1, ctl));
          if (!ok) break;
          clear_rows<2 + TN / 64 / CG>(smem + last * kStageBytes, valid, lane);
          if (lane == 0) mbar_arrive_release(cluster_addr(smem_u32(&s.full[last]), 0));
          phases ^= 1u << last;
          ++handed_on;
        }
        if (lane == 0) s.tails_done = handed_on;
      }
      __syncwarp();
    } else if (warp == 1) {
      Issuer<P, CG, TN, FP8, kAmn, kBmn> io(s, smem, tmem, ctl);
      bool ok = true;
      Tile t;
      while (ok && walk.next(t)) {
        const int blocks = __shfl_sync(~0u, t.kb, 0);  // uniform, and known to be
        const int tail = OP == kDw ? __shfl_sync(~0u, t.rows, 0) & 63 : 0;
        for (int kb = 0; kb < blocks; ++kb) {
          ok = io.wait(FP8 || kb == 0);
          if (!ok) break;
          int steps = 4;
          if (OP == kDw && tail != 0 && kb == blocks - 1) {
            // rows of the next segment follow: zero them in both operands
            steps = (tail + 15) >> 4;
            clear_rows<2 + TN / 64 / CG>(smem + io.st * kStageBytes, tail, lane);
          }
          io.block(FP8 || kb == 0, FP8 || kb == blocks - 1, steps);
        }
      }
      __syncwarp();
      tc_commit<CG>(smem_u32(&s.drain));  // products in flight end before TMEM is freed
      mbar_drain(smem_u32(&s.drain), 0);
      __syncwarp();
    } else if constexpr (FP8) {
      scale_warp<OP, CG>(p, s, ctl, walk, (warp - 2) * 32 + lane);
      __syncwarp();
    }
  } else {
    take_registers<FP8>();
    const int ew = warp - kEpiWarp0, quarter = warp & 3, half = ew >> 2;
    uint4* buf = epi + ew * (P::kWarpBytes / 16);
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    int as = 0;
    uint32_t aph = 0, parity = 0;
    bool ok = true;
    Tile t;
    while (ok && walk.next(t)) {
      if constexpr (!FP8) {
        GateUp pre;
        if constexpr (OP == kDgate) gate_fetch<TN>(pre, p, t, half, quarter, lane, 0);
        if (t.kb > 0) {
          ok = __all_sync(~0u, mbar_wait<kPair>(smem_u32(&s.tfull[as]), aph, ctl));
          if (!ok) break;
          tc_fence_after();
        }
        epilogue_bf16<OP, TN>(p, t, tmem + lanes + as * kAccColumns, half, quarter, lane, buf,
                              t.kb == 0, pre, map_c);
        if (t.kb > 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) release<CG>(s, as);
          as ^= 1;
          if (as == 0) aph ^= 1;
        }
      } else {
        // columns of this thread: kGated 64 of gate and the same 64 of up,
        // kDown 128 in a row of one weight block
        const int r = quarter * 32 + lane;
        const bool mine = r < t.rows;
        const uint32_t c0 = OP == kGated ? half * 64 : half * 128;
        const uint32_t c1 = OP == kGated ? 128 + half * 64 : half * 128 + 64;
        float2 acc[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = make_float2(0.0f, 0.0f);
        for (int kb = 0; kb < t.kb; ++kb) {
          ok = __all_sync(~0u, mbar_wait<kPair>(smem_u32(&s.tfull[as]), aph, ctl));
          if (!ok) break;
          tc_fence_after();
          const uint32_t ta = tmem + lanes + as * kAccColumns;
          uint32_t v[2][32];
          tc_ld32(v[0], ta + c0);
          const float2 sc = s.scale[as][r];
          const float s0 = OP == kGated || half == 0 ? sc.x : sc.y;
          const float s1 = OP == kGated ? sc.y : s0;
#pragma unroll
          for (int g = 0; g < 4; ++g) {  // the next 32 columns load beside this sum
            tc_wait_ld();
            tc_loaded(v[g & 1]);
            if (g < 3) {
              tc_ld32(v[(g + 1) & 1], ta + (g < 1 ? c0 + 32 : g < 2 ? c1 : c1 + 32));
            } else {  // all read: the accumulator and the scales may be overwritten
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                release<CG>(s, as);
                mbar_arrive(smem_u32(&s.sempty[as]));
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              fma2(acc[g * 16 + i], v[g & 1][2 * i], v[g & 1][2 * i + 1], g < 2 ? s0 : s1);
          }
          as ^= 1;
          if (as == 0) aph ^= 1;
        }
        if (!ok) break;
        const long long row = (long long)t.row0 + quarter * 32;
        if constexpr (OP == kDown) {
          // To the copy engine: stored by the lanes themselves, 32 rows at a time, a
          // tile's 64 KB take about 5500 cycles in which the products wait for the
          // registers. The few warps with a segment's end still store so.
          const int col = t.n0 * TN + half * 128;
          const int left = t.rows - quarter * 32;
          if (col < p.N && left >= 32) {
            out_begin(lane);
#pragma unroll
            for (int g = 0; g < 16; ++g)
              buf[out_unit(lane, g)] = make_uint4(bf16x2(acc[g * 4].x, acc[g * 4].y),
                                                  bf16x2(acc[g * 4 + 1].x, acc[g * 4 + 1].y),
                                                  bf16x2(acc[g * 4 + 2].x, acc[g * 4 + 2].y),
                                                  bf16x2(acc[g * 4 + 3].x, acc[g * 4 + 3].y));
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&map_c, smem_u32(buf), col, (int)row);
              tma_store_2d(&map_c, smem_u32(buf) + 4096, col + 64, (int)row);
              bulk_commit();
            }
          } else if (col < p.N && mine) {
            uint16_t* out = static_cast<uint16_t*>(p.out) + (row + lane) * p.N + col;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              uint32_t o[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = bf16x2(acc[g * 8 + i].x, acc[g * 8 + i].y);
              store32(out + g * 16, o);
            }
          }
        } else {
          // h = silu(g) u, then e4m3 codes with one scale for the tile's 128
          // columns of the row: its largest magnitude comes from this thread
          // and the one of the other half
          float h[64], m = 0.0f;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            h[2 * i] = silu(acc[i].x) * acc[32 + i].x;
            h[2 * i + 1] = silu(acc[i].y) * acc[32 + i].y;
            m = max_nan(m, max_nan(fabsf(h[2 * i]), fabsf(h[2 * i + 1])));
          }
          s.amax[parity][half][r] = m;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.pair[quarter]));
          ok = __all_sync(~0u, mbar_wait<kPair>(smem_u32(&s.pair[quarter]), parity, ctl));
          if (!ok) break;
          m = max_nan(m, s.amax[parity][half ^ 1][r]);
          parity ^= 1;  // the other buffer next: this one is read until then
          const float scale = __fdiv_rn(m, 448.0f);
          if (mine && half == 0) p.out_scale[((long long)t.row0 + r) * (p.F >> 7) + t.n0] = scale;
          uint8_t* out =
              static_cast<uint8_t*>(p.out) + (row + lane) * p.F + t.n0 * 128 + half * 64;
          // the reciprocal and its products far from underflow and overflow
          const bool quick = scale >= 0x1p-64f && scale <= 0x1p64f;
          const float y = quick ? __frcp_rn(scale) : 0.0f;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t q[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) {
              const float* f = h + 32 * u + 4 * w;
              if (quick) {
                const float2 a = minus_quotient(make_float2(f[0], f[1]), scale, y);
                const float2 b = minus_quotient(make_float2(f[2], f[3]), scale, y);
                q[w] = e4m3x4(a.x, a.y, b.x, b.y) ^ 0x80808080u;
              } else if (scale > 0.0f) {
                q[w] = e4m3x4(__fdiv_rn(f[0], scale), __fdiv_rn(f[1], scale),
                              __fdiv_rn(f[2], scale), __fdiv_rn(f[3], scale));
              } else {
                q[w] = 0u;
              }
            }
            if (mine) store32(out + u * 32, q);
          }
        }
      }
    }
    if constexpr (P::kOut) bulk_wait();  // the copies out of this CTA's memory are done
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (kPair) {
    cluster_sync();  // neither CTA's memory is used any more, unless a wait gave up
    if (*ctl.abort) {  // set in both CTAs before that
      if (warp == 0) settle_pair<OP, kStages>(s, rank);
      cluster_sync();
    }
  } else {
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 2) tc_dealloc<CG>(tmem, 512);
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
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
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

// Row tiles are at most one per `rows` rows plus one per segment; the host
// knows no more.
template <int OP>
long long most_tiles(const ExpertArgs& p, int rows, int nt) {
  if (OP == kDw) return (long long)((p.M + rows - 1) / rows) * nt * p.E;
  return (p.rows_max / rows + (p.E < p.rows_max ? p.E : p.rows_max)) * nt;
}

template <int OP>
int column_tiles(const ExpertArgs& p, int tn) {
  const int n = OP == kGated ? p.F : p.N, w = OP == kGated ? tn / 2 : tn;
  return (n + w - 1) / w;
}

template <int OP, bool FP8, int CG, int TN>
cudaError_t launch(const ExpertArgs& args, const void* a, const void* b, int num_sms,
                   cudaStream_t st) {
  constexpr int kRows = kTileM * CG;
  ExpertArgs p = args;
  p.nt = column_tiles<OP>(p, TN);
  // Segments of a few rows copy no more than those, 32 at a time.
  p.a_box = CG == 1 && p.rows_max <= 64ll * p.E ? 32 : 128;
  CUtensorMap ma, mb, mc = {};
  cudaError_t e;
  if (OP == kDw) {
    e = make_map(&ma, a, false, p.M, p.rows_max, 0, 64);
    if (e == cudaSuccess) e = make_map(&mb, b, false, p.N, p.rows_max, 0, 64);
  } else {
    e = make_map(&ma, a, FP8, p.K, p.rows_max, 0, p.a_box);
    if (e == cudaSuccess) {
      if (OP == kGated) e = make_map(&mb, b, FP8, p.K, 2ll * p.F, p.E, TN / 2);
      else if (OP == kDown) e = make_map(&mb, b, FP8, p.K, p.N, p.E, TN / 2);
      else e = make_map(&mb, b, false, p.N, p.K, p.E, 64);
    }
  }
  if (e == cudaSuccess && OP == kDw && TN == 128)
    e = make_map(&mc, p.out, false, p.N, p.M, p.E, 32);
  if (e == cudaSuccess && OP == kDown && FP8)
    e = make_map(&mc, p.out, false, p.N, p.rows_max, 0, 32);
  if (e != cudaSuccess) return e;
  const long long tiles = most_tiles<OP>(p, kRows, p.nt);
  const long long most = num_sms / CG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < most ? tiles : most) * CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<OP, FP8, CG, TN>();
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
  return cudaLaunchKernelEx(&cfg, k_expert_gemm<OP, FP8, CG, TN>, ma, mb, mc, p);
}

// Whether pairs of CTAs share 256-row tiles: each then writes and reads a
// third less of its shared memory per product, but an expert's last tile
// wastes up to 255 rows instead of 127. By average rows per expert (the host
// knows no others). Measured at E = 32, H = 4096, F = 2048, bf16, us alone /
// paired: kGated 192 / 192 at 128 rows, 221 / 194 at 192, 401 / 381 at 512,
// 734 / 663 at 1024; kDgate 120 / 138 at 128, 163 / 160 at 256; kDx 175 / 179
// at 128, 251 / 230 at 256; kDw, where the rows are the reduction axis and the
// epilogue of a short sum weighs more, 480 / 498 at 512, 757 / 737 at 1024.
// e4m3 (H = 7168) does not gain: 961 / 1158 at 512 rows, where an accumulator
// is handed back and forth between the two CTAs for each 128 channels. The rule
// does not look at how many tiles there are: alone / paired at 32768 rows of
// one expert, backward of H = 256, F = 128 327 / 341 (two weight tiles, each
// 512 blocks long), of H = 4096, F = 1408 1774 / 1515.
bool use_pair(ExpertOp op, bool fp8, const ExpertArgs& p) {
  if (fp8) return false;
  return p.rows_max >= (op == kDw ? 768ll : 192ll) * p.E;
}

// Whether tiles are 128 columns wide: where 256 would give at most two tiles
// per SM, more and smaller ones spread a product's copies, which bound it then,
// over more SMs (64 bytes a cycle go into each). bf16, uniform routing, passes
// one after another, tiles of 256 / 128 columns, us: backward of 231 rows,
// E = 16, H = 520, F = 264 39.8 / 30.4; H = 4096, F = 1408, E = 8: down at 1024
// rows 24.1 / 23.2, gated at 1400 58.9 / 55.1. What the rule gives away: where
// the wide tiles come to about whole turns of the SMs, narrow ones only add to
// the copies (there, gated at 512 rows 38.5 / 49.4, down 13.9 / 18.4, and at
// 1400 rows 25.5 / 29.3). Where tiles are many they cost: E = 16 at 2048 rows
// gated 70.4 / 77.1, down 41.1 / 45.1, backward 265 / 318; kDw of E = 32,
// H = 4096, F = 2048 at 512 rows an expert makes its backward pass 1316 / 1618.
template <int OP>
bool use_narrow(const ExpertArgs& p, int num_sms) {
  return most_tiles<OP>(p, kTileM, column_tiles<OP>(p, 256)) <= 2ll * num_sms;
}

template <int OP, bool FP8>
cudaError_t launch(bool pair, const ExpertArgs& p, const void* a, const void* b, int num_sms,
                   cudaStream_t st) {
  if constexpr (!FP8) {
    if (pair) return launch<OP, FP8, 2, 256>(p, a, b, num_sms, st);
    if (use_narrow<OP>(p, num_sms)) return launch<OP, FP8, 1, 128>(p, a, b, num_sms, st);
  }
  return launch<OP, FP8, 1, 256>(p, a, b, num_sms, st);
}

template <int OP, bool FP8, int CG, int TN>
cudaError_t prepare() {
  const auto kernel = k_expert_gemm<OP, FP8, CG, TN>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem_bytes<OP, FP8, CG, TN>());
  if (e != cudaSuccess || !FP8) return e;
  // The register split (4 warps x 56, 8 warps x 224) spends exactly 12 x 168.
  cudaFuncAttributes attr;
  e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return e;
  return attr.numRegs >= 168 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int OP, bool FP8>
cudaError_t prepare() {
  cudaError_t e = prepare<OP, FP8, 1, 256>();
  if constexpr (!FP8) {
    if (e == cudaSuccess) e = prepare<OP, FP8, 2, 256>();
    if (e == cudaSuccess) e = prepare<OP, FP8, 1, 128>();
  }
  return e;
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
  const bool pair = use_pair(op, fp8, p);
  switch (op) {
    case kGated:
      return fp8 ? launch<kGated, true>(pair, p, a, b, num_sms, st)
                 : launch<kGated, false>(pair, p, a, b, num_sms, st);
    case kDown:
      return fp8 ? launch<kDown, true>(pair, p, a, b, num_sms, st)
                 : launch<kDown, false>(pair, p, a, b, num_sms, st);
    case kDgate: return launch<kDgate, false>(pair, p, a, b, num_sms, st);
    case kDx: return launch<kDx, false>(pair, p, a, b, num_sms, st);
    default: return launch<kDw, false>(pair, p, a, b, num_sms, st);
  }
}

}  // namespace moe
