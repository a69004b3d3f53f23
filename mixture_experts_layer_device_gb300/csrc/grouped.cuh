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

}  // namespace moe
