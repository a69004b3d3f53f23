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
// How the tensor-core kernel cuts an expert's rows: as few tiles of up to `most`
// tokens (256; fewer in small calls) as hold them, all of one size (a multiple of 32)
// but the last.
constexpr int kTileTokens = 256;
MOE_DEV int tile_tokens(int rows, int most) {
  const int tiles = (rows + most - 1) / most;
  return ((rows + tiles - 1) / tiles + 31) & ~31;
}

// The tiles of a call: the experts that have rows in descending size of their
// tiles (eight classes of 32 tokens), an expert's tiles next to each other.
// Pairs that take tiles in turns then get equal work, and an expert's weights
// are read from memory once, by tiles that run at the same time.  (Whole tiles
// of all experts first and remainders last balanced no better and read the
// weights twice: 871 us against 855 at 32768 rows, 64 experts of [4096, 4096].)
//   off[E + 1]  the experts' clamped offsets
//   order[n]    the experts with rows, first[n + 1] their first tiles
struct TileTable {
  const int *off, *order, *first;
  int n, tiles;
};
inline __host__ __device__ int tile_table_ints(int E) { return 3 * E + 3; }
MOE_DEV TileTable tile_table_at(const int *p, int E) {
  TileTable t;
  t.off = p;
  t.order = p + E + 1;
  t.first = p + 2 * E + 1;
  t.n = p[3 * E + 2];
  t.tiles = t.first[t.n];
  return t;
}

// Builds the table at p by all THREADS threads of a block; `scratch`: 1 KB of shared
// memory.  No tiles at all when the offsets are bad (returns true).
template <int THREADS>
MOE_DEV bool build_tile_table(const GroupedArgs &g, int *p, int *scratch) {
  constexpr int W = THREADS / 32, CLASSES = 8;
  static_assert(W * CLASSES <= 256, "scratch");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = g.E;
  int *off = p, *order = p + E + 1, *first = p + 2 * E + 1;
  bool bad = false;
  for (int e = threadIdx.x; e < E; e += THREADS) {
    int lo, hi;
    bad |= !group_rows(g, e, lo, hi);
    off[e] = lo;
    if (e == E - 1) off[E] = hi;
  }
  const bool any = __syncthreads_or(bad);
  // A warp owns a run of consecutive experts: it counts their classes, and after
  // the warps' counts are summed (largest class first) places them in order.
  const int run = (E + W - 1) / W, from = warp * run, to = from + run < E ? from + run : E;
  int mine[CLASSES];
#pragma unroll
  for (int c = 0; c < CLASSES; ++c) mine[c] = 0;
  auto cls_of = [&](int e) {
    const int rows = e < to && !any ? off[e + 1] - off[e] : 0;
    return rows > 0 ? CLASSES - (tile_tokens(rows, g.most) >> 5) : -1;  // 0: the largest
  };
  for (int e0 = from; e0 < to; e0 += 32) {
    const int c = cls_of(e0 + lane);
#pragma unroll
    for (int k = 0; k < CLASSES; ++k) mine[k] += __popc(__ballot_sync(0xffffffffu, c == k));
  }
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < CLASSES; ++k) scratch[k * W + warp] = mine[k];
  __syncthreads();
  // every warp finds its first place in each class
  int at[CLASSES], total = 0;
#pragma unroll
  for (int k = 0; k < CLASSES; ++k) {
    int before = 0, all = 0;
    const int v = lane < W ? scratch[k * W + lane] : 0;
    before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
    all = __reduce_add_sync(0xffffffffu, v);
    at[k] = total + before;
    total += all;
  }
  for (int e0 = from; e0 < to; e0 += 32) {
    const int c = cls_of(e0 + lane);
#pragma unroll
    for (int k = 0; k < CLASSES; ++k) {
      const unsigned same = __ballot_sync(0xffffffffu, c == k);
      if (c == k) order[at[k] + __popc(same & ((1u << lane) - 1))] = e0 + lane;
      at[k] += __popc(same);
    }
  }
  __syncthreads();
  // first tiles along the order, by batches of THREADS experts
  int base = 0;
  for (int i0 = 0; i0 < total; i0 += THREADS) {
    const int i = i0 + threadIdx.x;
    int n = 0;
    if (i < total) {
      const int e = order[i], rows = off[e + 1] - off[e], size = tile_tokens(rows, g.most);
      n = (rows + size - 1) / size;
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    const int v = lane < W ? scratch[lane] : 0;
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
    if (i < total) first[i] = base + before + inc - n;
    base += __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    first[total] = base;
    p[3 * E + 2] = total;
  }
  __syncthreads();
  return any;
}

}  // namespace moe
