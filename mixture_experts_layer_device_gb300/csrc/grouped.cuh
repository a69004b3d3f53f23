// Shared by the grouped-product kernels: the rows of an expert.
#pragma once

#include "block.h"
#include "common.cuh"

namespace moe {

// Rows [lo, hi) of expert e, kept inside [0, rows] whatever the offsets hold;
// false when they descend or leave that range.
MOE_DEV bool group_rows(const GroupedArgs &g, int e, int &lo, int &hi) {
  const int a = __ldg(g.offsets + e), b = __ldg(g.offsets + e + 1);
  lo = a < 0 ? 0 : (a > g.rows ? g.rows : a);
  hi = b < lo ? lo : (b > g.rows ? g.rows : b);
  return a >= 0 && b >= a && b <= g.rows;
}

// Expert of tile u: the largest e with tiles[e] <= u (tiles ascends; experts
// without tiles repeat the value, so the last of them has the tile).
MOE_DEV int group_of_tile(const int *tiles, int E, int u) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tiles[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ---------------------------------------------------------------- token tiles
// How the tensor-core kernel cuts an expert's rows: whole tiles of 256 tokens,
// then what is left in one tile (up to 256 rows) or two equal ones.
constexpr int kTileTokens = 256;
struct TokenCut {
  int whole;  // whole tiles
  int rest;   // tiles of what is left: 0, 1 or 2
  int size;   // tokens of the first of them, a multiple of 32 when there are two
};
MOE_DEV TokenCut cut_tokens(int rows) {
  TokenCut c;
  if (rows <= kTileTokens) {
    c.whole = 0;
    c.rest = rows > 0 ? 1 : 0;
    c.size = rows;
  } else {
    c.whole = (rows - 1) / kTileTokens - 1;
    const int left = rows - c.whole * kTileTokens;  // 257 .. 512
    c.rest = 2;
    c.size = ((left + 1) / 2 + 31) & ~31;
  }
  return c;
}

// The tiles of a call in descending size: all whole ones by expert, then the
// others by size class (32 tokens each), so that tiles taken in turns cost
// every CTA pair the same.  Entry of `rest`: expert * 2 + which of its two.
// off: the experts' clamped offsets; whole[e]: whole tiles before expert e.
struct TileTable {
  int *off, *whole, *rest;
  int n_whole, n_rest;  // set by the builder
};
inline __host__ __device__ int tile_table_ints(int E) { return 4 * E + 4; }
MOE_DEV TileTable tile_table_at(int *p, int E) {
  TileTable t;
  t.off = p;
  t.whole = p + E + 1;
  t.rest = p + 2 * E + 2;
  t.n_whole = p[2 * E + 1];  // whole[E]
  t.n_rest = p[4 * E + 2];
  return t;
}

// Builds the table at p by all THREADS threads of a block; `scratch`: 256 bytes of
// shared memory.  No tiles at all when the offsets are bad (returns true).
template <int THREADS>
MOE_DEV bool build_tile_table(const GroupedArgs &g, int *p, unsigned long long *scratch) {
  constexpr int W = THREADS / 32;
  static_assert(W * 24 + 64 <= 1024, "scratch");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = g.E;
  int *off = p, *whole = p + E + 1, *rest = p + 2 * E + 2;
  bool bad = false;
  for (int e = threadIdx.x; e < E; e += THREADS) {
    int lo, hi;
    bad |= !group_rows(g, e, lo, hi);
    off[e] = lo;
    if (e == E - 1) off[E] = hi;
  }
  const bool any = __syncthreads_or(bad);
  // two passes: class totals, then places.  Eight classes in two words of four
  // 16-bit counters, which hold 2 E tiles.
  unsigned long long *tot = scratch + 3 * W;  // [2] totals of the classes, [1] of whole tiles
  unsigned long long base_a = 0, base_b = 0;  // first place of each class (after pass 0)
  for (int pass = 0; pass < 2; ++pass) {
    unsigned long long run_a = base_a, run_b = base_b;
    int run_w = 0;
    for (int from = 0; from < E; from += THREADS) {
      const int e = from + threadIdx.x;
      TokenCut c = {0, 0, 0};
      if (e < E && !any) c = cut_tokens(off[e + 1] - off[e]);
      const int cls = c.rest ? (c.size - 1) >> 5 : 0;  // 0 .. 7
      unsigned long long a = 0, b = 0;
      if (cls < 4) a = static_cast<unsigned long long>(c.rest) << (16 * cls);
      else b = static_cast<unsigned long long>(c.rest) << (16 * (cls - 4));
      unsigned long long ia = a, ib = b;
      int iw = c.whole;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long va = __shfl_up_sync(0xffffffffu, ia, o), vb = __shfl_up_sync(0xffffffffu, ib, o);
        const int vw = __shfl_up_sync(0xffffffffu, iw, o);
        if (lane >= o) {
          ia += va;
          ib += vb;
          iw += vw;
        }
      }
      if (lane == 31) {
        scratch[warp] = ia;
        scratch[W + warp] = ib;
        scratch[2 * W + warp] = static_cast<unsigned>(iw);
      }
      __syncthreads();
      for (int w = 0; w < W; ++w) {
        if (w < warp) {
          ia += scratch[w];
          ib += scratch[W + w];
          iw += static_cast<int>(scratch[2 * W + w]);
        }
      }
      if (pass == 1 && e < E) {
        whole[e] = run_w + iw - c.whole;
        if (c.rest) {
          const unsigned long long q = cls < 4 ? run_a + ia - a : run_b + ib - b;
          const int at = static_cast<int>((q >> (16 * (cls & 3))) & 0xFFFFu);
          rest[at] = 2 * e;
          if (c.rest == 2) rest[at + 1] = 2 * e + 1;
        }
      }
      // the running totals of the batch: the last thread has them all
      if (threadIdx.x == THREADS - 1) {
        tot[0] = run_a + ia;
        tot[1] = run_b + ib;
        tot[2] = static_cast<unsigned>(run_w + iw);
      }
      __syncthreads();
      run_a = tot[0];
      run_b = tot[1];
      run_w = static_cast<int>(tot[2]);
    }
    if (pass == 0) {
      // largest class first
      unsigned at = 0;
#pragma unroll
      for (int cls = 7; cls >= 0; --cls) {
        const unsigned n = static_cast<unsigned>(((cls < 4 ? run_a : run_b) >> (16 * (cls & 3))) & 0xFFFFu);
        if (cls < 4) base_a |= static_cast<unsigned long long>(at) << (16 * cls);
        else base_b |= static_cast<unsigned long long>(at) << (16 * (cls - 4));
        at += n;
      }
      if (threadIdx.x == 0) p[4 * E + 2] = at;
    } else if (threadIdx.x == 0) {
      whole[E] = run_w;
    }
    __syncthreads();
  }
  return any;
}

}  // namespace moe
