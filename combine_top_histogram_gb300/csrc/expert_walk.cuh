// expert_walk.cuh -- the segments of the experts' rows and the tiles of a
// product over them, as a persistent CTA (or pair of CTAs) takes them. Device
// code only.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "expert_internal.cuh"

namespace moe {

constexpr int kGroupM = 8;             // row tiles that share weight tiles in L2

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
// DW: kDw's tiles. ROWS: rows of a CTA's (or pair's) tile, of which this CTA's
// begin at row `part`. S: shared memory with off[E + 1], pre[E + 1] and, for kDw,
// uneven.
template <bool DW, int ROWS, class S>
struct Walk {
  static constexpr int kRows = ROWS;
  const ExpertArgs& p;
  const S& s;
  const int k_elems, part, first, step, mt_w;
  int t, e, base, per;  // tile, its expert, the expert's first tile and tiles
  int place = 0;        // kDw: the expert's place by falling rows
  bool uneven, back = true;  // kDw: some experts' rows are many more; this step goes backwards

  __device__ __forceinline__ Walk(const ExpertArgs& pa, const S& sh, int ke, int pt, int tile0,
                                  int st)
      : p(pa), s(sh), k_elems(ke), part(pt), first(tile0), step(st),
        mt_w(DW ? (pa.M + kRows - 1) / kRows : 0), t(tile0 - st), e(0), base(0) {
    per = tiles(0);
    uneven = false;
    if constexpr (DW) {
      uneven = sh.uneven;
      if (uneven) e = sh.pre[0];
    }
  }

  __device__ __forceinline__ int tiles(int x) const {
    return (DW ? mt_w : s.pre[x + 1] - s.pre[x]) * p.nt;
  }

  __device__ __forceinline__ bool next(Tile& o) {
    t += step;
    uint32_t local;  // tile of the expert
    if (DW) {
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
    const int mt = DW ? mt_w : s.pre[e + 1] - s.pre[e];
    const uint32_t group = kGroupM * p.nt;
    const uint32_t g = local / group, idx = local - g * group;
    const uint32_t gs = min(kGroupM, mt - (int)g * kGroupM);
    const uint32_t n = gs == kGroupM ? idx / kGroupM : idx / gs;
    const int m = (int)(g * kGroupM + idx - n * gs) * kRows + part;
    o.e = e;
    o.n0 = (int)n;
    if (DW) {
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
template <int ROWS, int THREADS, class S>
__device__ __forceinline__ void load_segments(const ExpertArgs& p, S& s) {
  for (int e = threadIdx.x; e <= p.E; e += THREADS) {
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
      const int tiles = (n + ROWS - 1) / ROWS;
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

}  // namespace moe
