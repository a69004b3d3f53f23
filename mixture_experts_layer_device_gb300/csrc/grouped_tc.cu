// Ragged grouped products on CTA pairs (tcgen05, cta_group::2).
//
// The tokens are the N side of the tensor-core product: y^T = w x^T with 256
// output features (M, 128 per CTA) by up to 256 tokens, and N is set per tile in
// steps of 32.  An expert's rows start and end anywhere, so with the tokens on
// M every expert would cost whole 128-row tiles; on N its last tile costs what
// it holds.  Rows past the expert's last one are computed with whatever lies
// there (another expert's rows) and not stored: a token is a column of its own.
//
//   forward   A = w [N, K] K-major             B = x K-major     columns: tokens
//   dgrad     A = w^T: w read MN-major         B = dy K-major    columns: tokens
//   gated     A = w's rows [gate 16 | up 16 | gate 16 ..] K-major, B = x: 128 features of h
//             per pair, both projections of a feature in one warp's 32 lanes
//   wgrad     A = dy^T, B = x^T: both read MN-major, the reduction runs over the
//             expert's rows.  Rows past its last one must not enter the sum
//             (0 * NaN is NaN), so each expert has its own pair of tensor maps
//             that end at its last row: TMA fills zeros beyond it.
//
// No operand is transposed in memory: the MN-major operands are 64 x 64 boxes
// (64 features wide, 64 reduction steps deep) in the 128-byte swizzle, which the
// shared-memory descriptors address directly.
//
// Roles per CTA (320 threads): TMA producer, MMA issuer (leader CTA), eight
// epilogue warps (two per quarter of the accumulator's rows: one alone works on
// its instructions' latencies); three 64 KB stages; two accumulators of 256 TMEM columns, so a
// tile's epilogue runs beside the next one's MMAs.  Persistent: pair c takes
// tiles c, c + pairs, ...  Every wait is bounded (mbar_wait).
#include <type_traits>

#include "elem.cuh"
#include "gate_act.cuh"
#include "gemm_common.cuh"
#include "grouped.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kBlockBytes = 32768;           // 64 reduction steps: 16 KB of A, up to 16 KB of B
constexpr int kThreads = 320;
constexpr int kEpilogueWarps = 8;
constexpr int kStaging = 4096;               // per epilogue warp

// Blocks per stage: 300 us where one takes 342 (16384 rows over four experts of [4096,
// 4096]).  Whether a stage's barriers or its loads' latency cost it is not measured.
constexpr int kBlocks = 2;
constexpr int kStages = 3;
constexpr int kStageBytes = kBlocks * kBlockBytes;
constexpr size_t kSmem = 1024 + kStages * kStageBytes + kEpilogueWarps * kStaging + (2 * kStages + 5) * 8 + 16;
static_assert(kSmem <= 232448, "shared memory");
// Forward and dgrad stage 2 KB per warp and keep the tile table in the rest of
// the staging; more experts than it holds take the plan launch's table.
constexpr int kTablePlace = kEpilogueWarps * 2048;
constexpr int kPairs = 76;
constexpr int kTableExperts = ((kEpilogueWarps * kStaging - kTablePlace) / 4 - 3) / 3;

struct TcMaps {
  CUtensorMap a;        // forward, dgrad: w
  CUtensorMap b[8];     // token rows, boxes of 16, 32, .. 128 rows
  CUtensorMap out;      // wgrad: dw
};

MOE_DEV void tma_load_3d_pair(const CUtensorMap *map, uint32_t mbar, void *dst, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(mbar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
MOE_DEV void tma_load_4d_pair(const CUtensorMap *map, uint32_t mbar, void *dst, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(mbar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
MOE_DEV void tma_load_5d_pair(const CUtensorMap *map, uint32_t mbar, void *dst, int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(mbar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
MOE_DEV void tma_store_3d(const CUtensorMap *map, const void *src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
MOE_DEV void tma_add_3d(const CUtensorMap *map, const void *src, int c0, int c1, int c2) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   map),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// Descriptor of an MN-major operand in the 128-byte swizzle: rows of 64 features
// (128 bytes), one per reduction step; 8 steps (1024 bytes) to the next group
// of 8, 64 steps (8192 bytes) to the next 64 features.
MOE_DEV uint64_t mn_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Instruction descriptor of kind::f16 with fp32 accumulation, M = 256 over the
// pair: operand format (1 bf16, 0 fp16) at [7,10) and [10,13), MN-major A / B at
// bits 15 / 16, N >> 3 at [17,23), M >> 4 at [24,29).
template <int DIR>
MOE_DEV uint32_t tc_idesc(int dtype, int n) {
  const uint32_t f = dtype == MOE_ELEM_BF16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | (DIR == GROUPED_DGRAD || DIR == GROUPED_WGRAD ? 1u << 15 : 0u) |
         (DIR == GROUPED_WGRAD ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (16u << 24);
}

// How many reduction steps one accumulator takes.  It truncates at every instruction, always
// towards zero: a chain of 16384 of them left a dw of terms of one sign (262144 rows of one
// expert) 4.3e-4 of its size too low.  CHAINS, for weight gradients of more rows than kChain in
// fp32, or than kChain16 in 16 bits: chains of 8192 steps joined in fp32 lose 2.5e-6, whatever
// the rows, at no cost; of 2048 2.2e-7, but 20000 rows of two experts of [1057, 2001] added to a
// given dw take 285 us instead of 250 (the next tile's product stops at a chain's end while
// elements leave); of 65536, in front of a rounding to 16 bits, 6.7e-5.
constexpr int kChain = 8192, kChain16 = 65536;
template <bool WIDE, bool CHAINS>
MOE_DEV int chain_of(int klen) {
  return CHAINS ? (WIDE ? kChain : kChain16) : (klen > 0 ? klen : 1);
}

MOE_DEV void tmem_ld16_async(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

struct TcTile {
  int e;
  int f0;     // first output feature of the pair (A's rows)
  int c0;     // first column: token row (forward, dgrad) or feature (wgrad)
  int n;      // columns of the product: a multiple of 32 (wgrad: 128)
  int valid;  // columns that are stored
  int k0;     // first reduction step (wgrad: the expert's first row)
  int klen;   // reduction length
};

// The tiles of a call in the order in which the pairs take them.
template <int DIR>
struct TcTiles {
  const GroupedArgs &g;
  TileTable t;
  int nf, nc, total;
  MOE_DEV TcTiles(const GroupedArgs &args, int *table) : g(args) {
    nf = DIR == GROUPED_GATED ? ((g.N >> 1) + 127) >> 7 : ((DIR == GROUPED_DGRAD ? g.K : g.N) + 255) >> 8;
    if constexpr (DIR == GROUPED_WGRAD) {
      nc = (g.K + 255) >> 8;
      total = (g.zeroed || g.accumulate ? __ldg(g.order + g.E) : g.E) * nf * nc;  // the experts without rows stand last
    } else {
      t = tile_table_at(table, g.E);
      nc = 1;
      total = t.tiles * nf;
    }
  }
  // The same without the end: whatever lies past it is not used.
  MOE_DEV TcTile ahead(int u) const { return u < total ? at(u) : TcTile(); }
  // Pair p's i-th tile: back and forth over the pairs, so that in a descending
  // order of sizes no pair always gets the larger one.
  MOE_DEV int unit(int i, int p, int pairs) const { return i * pairs + ((i & 1) ? pairs - 1 - p : p); }
  MOE_DEV TcTile at(int u) const {
    TcTile r;
    if constexpr (DIR == GROUPED_WGRAD) {
      const int per = nf * nc, q = u / per, w = u - q * per;
      r.e = __ldg(g.order + q);
      r.f0 = (w / nc) * 256;
      r.c0 = (w % nc) * 256;
      r.valid = g.K - r.c0 < 256 ? g.K - r.c0 : 256;
      // MN-major columns come in whole 64-feature blocks per CTA
      r.n = r.valid > 128 ? 256 : 128;
      int lo, hi;
      group_rows(g, r.e, lo, hi);
      r.k0 = lo;
      r.klen = hi - lo;
    } else {
      const int i = group_of_tile(t.first, t.n, u / nf);
      const int first = t.first[i], mt = t.first[i + 1] - first, local = u - first * nf;
      r.e = t.order[i];
      const int lo = t.off[r.e], rows = t.off[r.e + 1] - lo, size = tile_tokens(rows, g.most);
      r.f0 = (local / mt) * (DIR == GROUPED_GATED ? 128 : 256);
      const int from = (local % mt) * size;
      r.c0 = lo + from;
      r.valid = rows - from < size ? rows - from : size;
      r.n = (r.valid + 31) & ~31;
      r.k0 = 0;
      r.klen = DIR == GROUPED_DGRAD ? g.N : g.K;
    }
    return r;
  }
};

// A piece of 32 tokens x 32 features from one warp's accumulator columns (lane =
// feature): neighbouring lanes swap so that each holds two features of one
// token, and the piece leaves through shared memory as 16-byte stores.
template <typename T>
MOE_DEV void put_tokens(const float *v, uint8_t *buf, T *out, long ld, int tokens, int features, int lane) {
  const bool odd = lane & 1;
  __syncwarp();
#pragma unroll
  for (int t = 0; t < 32; t += 2) {
    const float mine = odd ? v[t + 1] : v[t];
    const float other = __shfl_xor_sync(0xffffffffu, odd ? v[t] : v[t + 1], 1);
    const uint32_t w = odd ? Elem<T>::pack2(other, mine) : Elem<T>::pack2(mine, other);
    *reinterpret_cast<uint32_t *>(buf + (t + (odd ? 1 : 0)) * 64 + (lane >> 1) * 4) = w;
  }
  __syncwarp();
  const int c = (lane & 3) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = (lane >> 2) + 8 * i;
    if (t < tokens && c < features)
      *reinterpret_cast<uint4 *>(out + t * ld + c) = *reinterpret_cast<const uint4 *>(buf + t * 64 + c * 2);
  }
}

// The same for a piece whose lanes 0 .. 15 hold 16 features of the gate and lanes 16 ..
// 31 those of the up projection: [g | u] of each token, `half` elements apart.
template <typename T>
MOE_DEV void put_gate_up(const float *v, uint8_t *buf, T *out, long ld, int half, int tokens, int features, bool vec, int lane) {
  if (!vec) {
#pragma unroll
    for (int t = 0; t < 32; ++t)
      if (t < tokens && (lane & 15) < features) out[t * ld + (lane < 16 ? lane : half + lane - 16)] = Elem<T>::from(v[t]);
    return;
  }
  const bool odd = lane & 1;
  __syncwarp();
#pragma unroll
  for (int t = 0; t < 32; t += 2) {
    const float mine = odd ? v[t + 1] : v[t];
    const float other = __shfl_xor_sync(0xffffffffu, odd ? v[t] : v[t + 1], 1);
    const uint32_t w = odd ? Elem<T>::pack2(other, mine) : Elem<T>::pack2(mine, other);
    *reinterpret_cast<uint32_t *>(buf + (t + (odd ? 1 : 0)) * 64 + (lane >> 1) * 4) = w;
  }
  __syncwarp();
  const int c = (lane & 1) * 8;
  T *to = out + ((lane & 2) ? half : 0) + c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = (lane >> 2) + 8 * i;
    if (t < tokens && c < features)
      *reinterpret_cast<uint4 *>(to + t * ld) = *reinterpret_cast<const uint4 *>(buf + t * 64 + (lane & 3) * 16);
  }
}

// h = act(g) u of that piece: a gate's lane and its up projection's, 16 apart, swap half of
// their tokens, so that each has both for 16 of them (even ones below lane 16, odd ones above).
template <typename T>
MOE_DEV void put_gated(const float *v, uint8_t *buf, T *out, long ld, int act, int tokens, int features, bool vec, int lane) {
  const bool up = lane & 16;
  float gate[16], h[16];
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    const float other = __shfl_xor_sync(0xffffffffu, up ? v[2 * t] : v[2 * t + 1], 16);
    gate[t] = up ? other : v[2 * t];
    h[t] = up ? v[2 * t + 1] : other;
  }
  switch (act) {
    case MOE_ACT_SILU:
#pragma unroll
      for (int t = 0; t < 16; ++t) h[t] *= act_value<MOE_ACT_SILU>(gate[t]);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int t = 0; t < 16; ++t) h[t] *= act_value<MOE_ACT_GELU>(gate[t]);
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int t = 0; t < 16; ++t) h[t] *= act_value<MOE_ACT_GELU_TANH>(gate[t]);
      break;
    default:
#pragma unroll
      for (int t = 0; t < 16; ++t) h[t] *= act_value<MOE_ACT_RELU>(gate[t]);
  }
  const int f = lane & 15, first = up ? 1 : 0;
  if (!vec) {
#pragma unroll
    for (int t = 0; t < 16; ++t)
      if (2 * t + first < tokens && f < features) out[(2 * t + first) * ld + f] = Elem<T>::from(h[t]);
    return;
  }
  __syncwarp();
#pragma unroll
  for (int t = 0; t < 16; ++t) *reinterpret_cast<T *>(buf + (2 * t + first) * 32 + f * 2) = Elem<T>::from(h[t]);
  __syncwarp();
  const int c = (lane & 1) * 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int t = (lane >> 1) + 16 * i;
    if (t < tokens && c < features)
      *reinterpret_cast<uint4 *>(out + t * ld + c) = *reinterpret_cast<const uint4 *>(buf + t * 32 + c * 2);
  }
}

// A piece of 32 rows x 128 bytes of dw (lane = row) into 128-byte-swizzled shared
// memory and out by TMA (or added to what is there), which clips it to the
// expert's matrix.  (As 16-byte stores of the lanes instead: 572 us where this is 506,
// 8192 rows and 128 experts of [2048, 4096].  A second buffer per warp in place of
// the third stage: 809 us where this is 768, 32768 skewed rows, 64 of [7168, 2048].)
MOE_DEV void put_rows(const uint32_t *w, uint8_t *buf, const CUtensorMap *map, bool add, int col, int row, int e, int lane) {
  if (lane == 0) bulk_wait_read<0>();  // the last piece has left the buffer
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4 *>(buf + lane * 128 + ((j ^ (lane & 7)) * 16)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (add) tma_add_3d(map, buf, col, row, e);
    else tma_store_3d(map, buf, col, row, e);
    bulk_commit();
  }
}

// The same piece element by element, for matrices whose rows are no whole 16-byte
// pieces: each store takes neighbouring columns of one row.
template <typename O>
MOE_DEV void put_elements(const uint32_t *w, uint8_t *buf, O *out, long ld, int rows, int cols, bool add, int lane) {
  constexpr int COLS = 128 / sizeof(O);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4 *>(buf + lane * 128 + ((j ^ (lane & 7)) * 16)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  __syncwarp();
  for (int r = 0; r < 32 && r < rows; ++r)
#pragma unroll
    for (int c = lane; c < COLS; c += 32) {
      const int byte = c * static_cast<int>(sizeof(O));
      const O v = *reinterpret_cast<const O *>(buf + r * 128 + (((byte >> 4) ^ (r & 7)) * 16) + (byte & 15));
      if (c < cols) {
        if constexpr (sizeof(O) == 4) out[r * ld + c] = add ? out[r * ld + c] + v : v;
        else out[r * ld + c] = v;
      }
    }
}

// T: the operands' type; WIDE: fp32 output (y or dw); CHAINS: dw from several accumulators.
template <int DIR, typename T, bool WIDE, bool CHAINS>
__global__ void __launch_bounds__(kThreads, 1) grouped_tc_kernel(const __grid_constant__ TcMaps maps, const GroupedArgs g) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  uint8_t *staging = smem + kStages * kStageBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(staging + kEpilogueWarps * kStaging);
  uint64_t *empty = full + kStages;
  uint64_t *tfull = empty + kStages;
  uint64_t *tempty = tfull + 2;
  uint64_t *done = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpilogueWarps);  // epilogue warps of both CTAs
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  int *table = g.tiles;
  if constexpr (DIR != GROUPED_WGRAD) {
    if (g.E <= kTableExperts) {
      table = reinterpret_cast<int *>(staging + kTablePlace);
      const bool bad = build_tile_table<kThreads>(g, table, reinterpret_cast<int *>(staging));
      if (blockIdx.x == 0 && threadIdx.x == 0) *g.status = bad ? kStatusBounds : 0;
    }
  }
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const TcTiles<DIR> tiles(g, table);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t ph = 0;
      int fenced = -1;
      TcTile next = tiles.ahead(pair);  // looked up one tile early: the look-up is a chain of loads
      for (int i = 0; tiles.unit(i, pair, pairs) < tiles.total && !*abort_flag; ++i) {
        const TcTile t = next;
        next = tiles.ahead(tiles.unit(i + 1, pair, pairs));
        const int half = t.n >> 1;
        const int fr = t.f0 + static_cast<int>(rank) * 128, cr = t.c0 + static_cast<int>(rank) * half;
        // a box of just the CTA's tokens: one request costs less than several that make
        // it up (32768 rows, 64 experts of [4096, 4096]: 811 us with boxes of 16, 32, 64
        // or 128 rows, 855 with sums of them)
        const int level = (half >> 4) - 1;
        const uint32_t b_bytes = DIR == GROUPED_WGRAD ? (half > 64 ? 16384u : 8192u) : 128u * static_cast<uint32_t>(half);
        const CUtensorMap *ma = &maps.a, *mb = &maps.b[level];
        if constexpr (DIR == GROUPED_WGRAD) {
          if (t.klen == 0) continue;
          ma = reinterpret_cast<const CUtensorMap *>(g.maps + static_cast<long>(t.e) * 256);
          mb = reinterpret_cast<const CUtensorMap *>(g.maps + static_cast<long>(t.e) * 256 + 128);
          if (fenced != t.e) {  // the maps were written by an earlier launch
            asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(ma) : "memory");
            asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(mb) : "memory");
            fenced = t.e;
          }
        }
        bool ok = true;
        for (int kb = 0; kb < t.klen; kb += 64 * kBlocks) {
          if (!mbar_wait(&empty[stage], ph ^ 1u, abort_flag, g.status)) {
            ok = false;
            break;
          }
          const int blocks = t.klen - kb > 64 ? kBlocks : 1;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2u * blocks * (16384u + b_bytes));
          const uint32_t bar = peer_smem(smem_u32(&full[stage]), 0);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            if (b >= blocks) break;
            uint8_t *sa = smem + stage * kStageBytes + b * kBlockBytes, *sb = sa + 16384;
            const int k = t.k0 + kb + 64 * b;
            if constexpr (DIR == GROUPED_FWD) {
              tma_load_3d_pair(ma, bar, sa, k, fr, t.e);
              tma_load_2d_pair(mb, bar, sb, k, cr);
            } else if constexpr (DIR == GROUPED_GATED) {
              const int f = t.f0 + static_cast<int>(rank) * 64;
              if (g.by_16) {
                tma_load_5d_pair(ma, bar, sa, k, 0, 0, f >> 4, t.e);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) tma_load_4d_pair(ma, bar, sa + i * 4096, k, f + 16 * i, 0, t.e);
              }
              tma_load_2d_pair(mb, bar, sb, k, cr);
            } else if constexpr (DIR == GROUPED_DGRAD) {
              tma_load_3d_pair(ma, bar, sa, fr, k, t.e);
              tma_load_3d_pair(ma, bar, sa + 8192, fr + 64, k, t.e);
              tma_load_2d_pair(mb, bar, sb, k, cr);
            } else {
              tma_load_2d_pair(ma, bar, sa, fr, k);
              tma_load_2d_pair(ma, bar, sa + 8192, fr + 64, k);
              tma_load_2d_pair(mb, bar, sb, cr, k);
              if (half > 64) tma_load_2d_pair(mb, bar, sb + 8192, cr + 64, k);
            }
          }
          if (++stage == kStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (pair leader)
    if (leader && lane == 0) {
      int stage = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      TcTile next = tiles.ahead(pair);
      for (int i = 0; tiles.unit(i, pair, pairs) < tiles.total && ok; ++i) {
        const TcTile t = next;
        next = tiles.ahead(tiles.unit(i + 1, pair, pairs));
        if (t.klen == 0) continue;
        const uint32_t idesc = tc_idesc<DIR>(g.dtype, t.n);
        for (int from = 0, chain = chain_of<WIDE, CHAINS>(t.klen); from < t.klen && ok; from += chain) {
          const int to = t.klen - from < chain ? t.klen : from + chain;
          if (!mbar_wait(&tempty[acc], aph ^ 1u, abort_flag, g.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t dt = tmem + static_cast<uint32_t>(acc * 256);
          for (int kb = from; kb < to; kb += 64 * kBlocks) {
            if (!mbar_wait(&full[stage], ph, abort_flag, g.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa0 = smem_u32(smem + stage * kStageBytes);
            const int left = to - kb;  // steps past the end hold zeros in both operands
#pragma unroll
            for (int k = 0; k < 4 * kBlocks; ++k) {
              if (k * 16 < left) {
                const uint32_t sa = sa0 + (k >> 2) * kBlockBytes, sb = sa + 16384;
                const uint64_t ad = DIR == GROUPED_FWD || DIR == GROUPED_GATED ? sw128_desc(sa + 32 * (k & 3))
                                                                                : mn_desc(sa + 2048 * (k & 3));
                const uint64_t bd = DIR == GROUPED_WGRAD ? mn_desc(sb + 2048 * (k & 3)) : sw128_desc(sb + 32 * (k & 3));
                mma_bf16_pair(dt, ad, bd, idesc, (kb - from | k) ? 1u : 0u);
              }
            }
            mma_commit_pair_mc(&empty[stage], 3);
            if (++stage == kStages) {
              stage = 0;
              ph ^= 1u;
            }
          }
          if (!ok) break;
          mma_commit_pair_mc(&tfull[acc], 3);
          if (++acc == 2) {
            acc = 0;
            aph ^= 1u;
          }
        }
      }
      mma_commit_pair_mc(done, 1);
      volatile int no_abort = 0;
      mbar_wait(done, 0, &no_abort, g.status);
    }
  } else {
    // ------------------------------------------------ epilogue (warps 2..9, both CTAs)
    const int q = warp & 3, half = (warp - 2) >> 2;  // accumulator rows; which of the pieces of 32 columns
    uint8_t *buf = staging + (warp - 2) * (DIR == GROUPED_WGRAD ? kStaging : 2048);
    int acc = 0;
    uint32_t aph = 0;
    if constexpr (DIR != GROUPED_WGRAD) {
      // zeros for the rows of no expert (the plan launch has done it otherwise)
      int lo, hi, lo_last, hi_last;
      group_rows(g, 0, lo, hi);
      group_rows(g, g.E - 1, lo_last, hi_last);
      const int outside = g.E <= kTableExperts ? lo + (g.rows - hi_last) : 0;
      const auto zero = [&](void *to, long ld, int bytes, bool vec) {
        uint8_t *out = static_cast<uint8_t *>(to);
        for (long i = blockIdx.x; i < outside; i += gridDim.x) {
          uint8_t *row = out + (i < lo ? i : hi_last + (i - lo)) * ld;
          if (vec) {
            for (int b = (threadIdx.x - 64) * 16; b < bytes; b += 32 * kEpilogueWarps * 16)
              *reinterpret_cast<uint4 *>(row + b) = make_uint4(0, 0, 0, 0);
          } else {
            for (int b = (threadIdx.x - 64) * 2; b < bytes; b += 32 * kEpilogueWarps * 2) *reinterpret_cast<uint16_t *>(row + b) = 0;
          }
        }
      };
      if constexpr (DIR == GROUPED_GATED) {
        zero(g.h, g.ld_h * 2, g.N, g.vec_h);
        if (g.y) zero(g.y, g.ld_y * 2, g.N * 2, g.vec_out);
      } else {
        zero(DIR == GROUPED_DGRAD ? g.dx : g.y, (DIR == GROUPED_DGRAD ? g.ld_x : g.ld_y) * (WIDE ? 4 : 2),
             (DIR == GROUPED_DGRAD ? g.K : g.N) * (WIDE ? 4 : 2), g.vec_out);
      }
    }
    if (DIR == GROUPED_DGRAD && g.chained && warp == 2) {
      pdl_wait();  // the maps are written: the weight gradient may start where an SM is free
      pdl_trigger();
    }
    TcTile next = tiles.ahead(pair);
    for (int i = 0; tiles.unit(i, pair, pairs) < tiles.total; ++i) {
      const TcTile t = next;
      next = tiles.ahead(tiles.unit(i + 1, pair, pairs));
      const int fr = t.f0 + static_cast<int>(rank) * 128 + q * 32;  // this warp's first feature
      uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * 256);
      if (t.klen > 0) {
        if (!mbar_wait(&tfull[acc], aph, abort_flag, g.status)) break;
        tc_fence_after();
      }
      // one arrival per warp, without an order of its own at cluster scope: one per thread that
      // had it took the other CTA's warps some 1600 cycles a tile (60 experts of 128 rows, [4096,
      // 7168]: the weight gradient 843 us, 567 so)
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(&tempty[acc]);
          else mbar_arrive_remote_tmem(peer_smem(smem_u32(&tempty[acc]), 0));
        }
      };
      bool held = t.klen > 0;  // this warp has not released the accumulator yet
      if constexpr (DIR == GROUPED_WGRAD) {
        constexpr int STEP = WIDE ? 32 : 64;  // columns of a 128-byte piece
        if (CHAINS && t.klen > chain_of<WIDE, CHAINS>(t.klen)) {
          // the chains' sums meet in registers and go back to the last one's columns (kept in
          // registers up to the stores they would spill)
          bool lost = false;
          float z[128];
#pragma unroll
          for (int i = 0; i < 128; ++i) z[i] = 0.f;
          for (int from = 0, chain = chain_of<WIDE, CHAINS>(t.klen); from < t.klen; from += chain) {
            if (from > 0) {
              release();
              if (++acc == 2) {
                acc = 0;
                aph ^= 1u;
              }
              if (!mbar_wait(&tfull[acc], aph, abort_flag, g.status)) {
                lost = true;
                break;
              }
              tc_fence_after();
              tb = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * 256);
            }
#pragma unroll
            for (int j = 0; j < 128; j += 16) {
              const int col = (half + j / STEP * 2) * STEP + j % STEP;
              if (col >= t.n) continue;
              uint32_t more[16];
              tmem_ld16_async(tb + col, more);
              tmem_ld_wait();
              reg_fence<16>(more);
#pragma unroll
              for (int i = 0; i < 16; ++i) z[j + i] += __uint_as_float(more[i]);
            }
          }
          if (lost) break;
#pragma unroll
          for (int j = 0; j < 128; j += 32) {
            const int col = (half + j / STEP * 2) * STEP + j % STEP;
            if (col < t.n) tmem_st32(tb + col, reinterpret_cast<const uint32_t *>(z) + j);
          }
          tmem_st_wait();
        }
        for (int j = half * STEP; j < t.n; j += 2 * STEP) {
          uint32_t r[STEP], w[32];
          if (t.klen > 0) {
            tmem_ld32_async(tb + j, r);
            if (!WIDE) tmem_ld32_async(tb + j + 32, r + STEP - 32);
            tmem_ld_wait();
            reg_fence<STEP>(r);
          } else {
#pragma unroll
            for (int i = 0; i < STEP; ++i) r[i] = 0;
          }
          if (held && j + 2 * STEP >= t.n) {
            release();
            held = false;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if constexpr (WIDE) w[i] = r[i];
            else w[i] = Elem<T>::pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
          if (fr >= g.N || t.c0 + j >= g.K) continue;
          if (g.vec_out) {
            put_rows(w, buf, &maps.out, WIDE && g.accumulate, t.c0 + j, fr, t.e, lane);
          } else {
            using O = typename std::conditional<WIDE, float, T>::type;
            put_elements<O>(w, buf, static_cast<O *>(g.dw) + (static_cast<long>(t.e) * g.N + fr) * g.K + t.c0 + j, g.K,
                            g.N - fr, g.K - t.c0 - j, g.accumulate != 0, lane);
          }
        }
      } else if constexpr (DIR == GROUPED_GATED) {
        const int half_n = g.N >> 1, f = t.f0 + static_cast<int>(rank) * 64 + q * 16;  // this warp's first feature of h
        for (int j = half * 32; j < t.n; j += 64) {
          uint32_t r[32];
          tmem_ld32_async(tb + j, r);
          tmem_ld_wait();
          reg_fence<32>(r);
          if (j + 64 >= t.n) {
            release();
            held = false;
          }
          const int tokens = t.valid - j;
          if (f >= half_n) continue;
          const float *v = reinterpret_cast<const float *>(r);
          const long row = t.c0 + j;
          if (g.y)
            put_gate_up<T>(v, buf, static_cast<T *>(g.y) + row * g.ld_y + f, g.ld_y, half_n, tokens, half_n - f, g.vec_out, lane);
          put_gated<T>(v, buf, static_cast<T *>(g.h) + row * g.ld_h + f, g.ld_h, g.act, tokens, half_n - f, g.vec_h, lane);
        }
      } else {
        const int F = DIR == GROUPED_DGRAD ? g.K : g.N;
        const long ld = DIR == GROUPED_DGRAD ? g.ld_x : g.ld_y;
        for (int j = half * 32; j < t.n; j += 64) {
          uint32_t r[32];
          tmem_ld32_async(tb + j, r);
          tmem_ld_wait();
          reg_fence<32>(r);
          if (j + 64 >= t.n) {
            release();
            held = false;
          }
          const float *v = reinterpret_cast<const float *>(r);
          const long row = t.c0 + j;
          const int tokens = t.valid - j;
          if (fr >= F) continue;
          if constexpr (WIDE) {
            float *out = static_cast<float *>(g.y) + row * ld + fr + lane;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < tokens && fr + lane < F) out[i * ld] = v[i];
          } else {
            T *out = static_cast<T *>(DIR == GROUPED_DGRAD ? g.dx : g.y) + row * ld + fr;
            if (g.vec_out) {
              put_tokens(v, buf, out, ld, tokens, F - fr, lane);
            } else {  // rows that are no whole 16-byte pieces: 32 features of a token per store
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i < tokens && fr + lane < F) out[i * ld + lane] = Elem<T>::from(v[i]);
            }
          }
        }
      }
      if (held) release();  // a narrow tile has no piece for this half
      if (t.klen > 0 && ++acc == 2) {
        acc = 0;
        aph ^= 1u;
      }
    }
    if (DIR == GROUPED_WGRAD && g.vec_out && lane == 0) bulk_wait<0>();
    if (DIR == GROUPED_WGRAD && g.chained && warp == 2) pdl_wait();  // the call ends with both gradients
  }

  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Before the weight gradient, by its last block the experts in descending order of
// rows (by buckets, an eighth of an octave wide), by the others their tensor maps:
// dy's and x's with the row extent cut to the expert's last row.  One warp per
// map; the copy to global memory makes it visible to later TMA accesses.
constexpr int kBuckets = 256;
MOE_DEV int size_bucket(int rows) {  // descending
  if (rows <= 0) return kBuckets - 1;
  const unsigned f = __float_as_uint(static_cast<float>(rows));
  const int b = static_cast<int>((f >> 20) - (127u << 3));  // eight steps per octave: 0 .. 247
  return kBuckets - 2 - b;
}
__global__ void __launch_bounds__(128) grouped_maps_kernel(const __grid_constant__ CUtensorMap dy,
                                                           const __grid_constant__ CUtensorMap x, const GroupedArgs g) {
  __shared__ __align__(128) uint32_t sm[4][32];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == gridDim.x - 1) {
    __shared__ int count[kBuckets];
    for (int i = threadIdx.x; i < kBuckets; i += 128) count[i] = 0;
    __syncthreads();
    bool bad = false;
    int lo, hi;
    for (int e = threadIdx.x; e < g.E; e += 128) {
      bad |= !group_rows(g, e, lo, hi);
      atomicAdd(&count[size_bucket(hi - lo)], 1);
    }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0 && !g.dx) *g.status = any ? kStatusBounds : 0;  // the call's first launch
    if (warp == 0) {
      int run = 0;
      for (int i = 0; i < kBuckets; i += 32) {
        const int v = count[i + lane];
        int inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int n = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += n;
        }
        count[i + lane] = run + inc - v;
        if (i + lane == kBuckets - 1) g.order[g.E] = run + inc - v;  // experts that have rows
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    __syncthreads();
    // places inside a bucket do not matter: an expert's tiles are computed alike wherever they stand
    for (int e = threadIdx.x; e < g.E; e += 128) {
      group_rows(g, e, lo, hi);
      g.order[atomicAdd(&count[size_bucket(hi - lo)], 1)] = e;
    }
    return;
  }
  const int i = blockIdx.x * 4 + warp;
  if (i >= 2 * g.E) return;
  sm[warp][lane] = reinterpret_cast<const uint32_t *>((i & 1) ? &x : &dy)[lane];
  __syncwarp();
  if (lane == 0) {
    int lo, hi;
    group_rows(g, i >> 1, lo, hi);
    const uint64_t at = smem_u32(sm[warp]);
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"l"(at), "r"(hi > 0 ? hi : 1)
                 : "memory");
  }
  __syncwarp();
  asm volatile(
      "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
          g.maps + static_cast<long>(i) * 128),
      "r"(smem_u32(sm[warp]))
      : "memory");
}

template <int DIR, typename T, bool WIDE, bool CHAINS>
int tc_clusters_query() {
  const auto kernel = grouped_tc_kernel<DIR, T, WIDE, CHAINS>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kSmem)) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
}

template <int DIR, typename T, bool WIDE, bool CHAINS>
cudaError_t launch_tc_kernel(const TcMaps &maps, const GroupedArgs &g, long units, cudaStream_t s) {
  static int memo[64] = {};
  const int most = per_device_memo(memo, tc_clusters_query<DIR, T, WIDE, CHAINS>);
  if (most <= 0) return cudaErrorInvalidConfiguration;
  if (units <= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * static_cast<unsigned>(units < most ? units : most), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g.chained ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, grouped_tc_kernel<DIR, T, WIDE, CHAINS>, maps, g);
}

// CHAINS costs registers, and some time where there is one chain (32768 rows, 64 experts of
// [4096, 4096], 16 bits: weight gradient 848 us, 815 without).
template <int DIR, typename T, bool WIDE>
cudaError_t launch_tc_one(const TcMaps &maps, const GroupedArgs &g, long units, cudaStream_t s) {
  if constexpr (DIR == GROUPED_WGRAD) {
    if (g.rows > (WIDE ? kChain : kChain16)) return launch_tc_kernel<DIR, T, WIDE, true>(maps, g, units, s);
  }
  return launch_tc_kernel<DIR, T, WIDE, false>(maps, g, units, s);
}

template <int DIR>
cudaError_t launch_tc(const TcMaps &maps, const GroupedArgs &g, long units, cudaStream_t s) {
  const bool bf = g.dtype == MOE_ELEM_BF16;
  if constexpr (DIR == GROUPED_FWD || DIR == GROUPED_WGRAD) {
    if (g.out_dtype == MOE_ELEM_FP32)
      return bf ? launch_tc_one<DIR, __nv_bfloat16, true>(maps, g, units, s) : launch_tc_one<DIR, __half, true>(maps, g, units, s);
  }
  return bf ? launch_tc_one<DIR, __nv_bfloat16, false>(maps, g, units, s) : launch_tc_one<DIR, __half, false>(maps, g, units, s);
}

// Token rows [rows, cols] with boxes of 64 columns x 16 (i + 1) rows.
bool row_maps(CUtensorMap *m, int elem, const void *p, long rows, int cols, long ld) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(ld) * 2};
  for (int i = 0; i < 8; ++i) {
    const uint32_t box[2] = {64, 16u * (i + 1)};
    if (!host_encode_map(&m[i], elem, p, 2, dims, strides, box)) return false;
  }
  return true;
}

bool expert_map(CUtensorMap *m, int elem, const void *p, const GroupedArgs &g, long ld, long ld_e, uint32_t c, uint32_t r) {
  const uint64_t e = elem_bytes(elem);
  const uint64_t dims[3] = {static_cast<uint64_t>(g.K), static_cast<uint64_t>(g.N), static_cast<uint64_t>(g.E)};
  const uint64_t strides[2] = {static_cast<uint64_t>(ld) * e, static_cast<uint64_t>(ld_e) * e};
  const uint32_t box[3] = {c, r, 1};
  return host_encode_map(m, elem, p, 3, dims, strides, box);
}

// w's rows as (column, 16 rows, gate or up, group of 16, expert), so that one box is 16 rows
// of the gate, the same 16 of the up projection, and so on; where m is no multiple of 16
// as (column, row, gate or up, expert), whose extent ends each projection, in boxes of
// one group.
bool gated_map(CUtensorMap *m, const GroupedArgs &g) {
  const uint64_t k = g.K, half = g.N / 2, row = static_cast<uint64_t>(g.ld_w) * 2, e = static_cast<uint64_t>(g.ld_e) * 2;
  if (g.by_16) {
    const uint64_t dims[5] = {k, 16, 2, half / 16, static_cast<uint64_t>(g.E)};
    const uint64_t strides[4] = {row, half * row, 16 * row, e};
    const uint32_t box[5] = {64, 16, 2, 4, 1};
    return host_encode_map(m, g.dtype, g.w, 5, dims, strides, box);
  }
  const uint64_t dims[4] = {k, half, 2, static_cast<uint64_t>(g.E)};
  const uint64_t strides[3] = {row, half * row, e};
  const uint32_t box[4] = {64, 16, 2, 1};
  return host_encode_map(m, g.dtype, g.w, 4, dims, strides, box);
}

// Where the rows of no expert and the tile table are made by a launch of their own.
cudaError_t plan_first(const GroupedArgs &g, int dir, cudaStream_t s) {
  if (g.E <= kTableExperts) return cudaSuccess;
  if (dir == GROUPED_GATED) {
    const cudaError_t e = g.y ? launch_grouped_plan(g, 0, g.y, g.dtype, g.N, g.ld_y, s) : cudaSuccess;
    return e == cudaSuccess ? launch_grouped_plan(g, 0, g.h, g.dtype, g.N >> 1, g.ld_h, s) : e;
  }
  const bool fwd = dir == GROUPED_FWD;
  return launch_grouped_plan(g, 0, fwd ? g.y : g.dx, fwd ? g.out_dtype : g.dtype, fwd ? g.N : g.K, fwd ? g.ld_y : g.ld_x, s);
}

bool wgrad_maps(const GroupedArgs &g, CUtensorMap *dy, CUtensorMap *x) {
  const uint64_t n[2] = {static_cast<uint64_t>(g.N), static_cast<uint64_t>(g.rows)};
  const uint64_t k[2] = {static_cast<uint64_t>(g.K), static_cast<uint64_t>(g.rows)};
  const uint64_t sn[1] = {static_cast<uint64_t>(g.in_y) * 2}, sk[1] = {static_cast<uint64_t>(g.in_x) * 2};
  const uint32_t box[2] = {64, 64};
  return host_encode_map(dy, g.dtype, g.dy, 2, n, sn, box) && host_encode_map(x, g.dtype, g.x, 2, k, sk, box);
}

cudaError_t launch_maps(const GroupedArgs &g, cudaStream_t s) {
  CUtensorMap dy, x;
  if (!wgrad_maps(g, &dy, &x)) return cudaErrorInvalidValue;
  HostTrace t("grouped_maps", s);
  grouped_maps_kernel<<<(2 * g.E + 3) / 4 + 1, 128, 0, s>>>(dy, x, g);
  return cudaGetLastError();
}

// Tiles of fewer tokens where even they all run in one round over the SM pairs: the
// reduction's length bounds a small call, and half a tile takes half of it (gated forward,
// 1500 rows of [256, 128]: 8.1 us, 12.6 with tiles of 256; 2043 rows, 8 experts of [512,
// 768]: 12.8 and 15.7).  Not where the weight gradient runs beside the data gradient on the
// pairs that it leaves (2043 rows of [3074, 768]: 42 us both, 30 with tiles of 256), and not
// where the plan launch has made the table, with tiles of 256.  An element's sum is the
// same in any tile.
int most_tokens(const GroupedArgs &g, int dir) {
  const long features = dir == GROUPED_GATED ? (g.N / 2 + 127) / 128 : ((dir == GROUPED_DGRAD ? g.K : g.N) + 255) / 256;
  const long experts = g.E < g.rows ? g.E : g.rows;
  int most = kTileTokens;
  while (!g.chained && g.E <= kTableExperts && most > 64 && ((g.rows + most / 2 - 1L) / (most / 2) + experts) * features <= kPairs) most /= 2;
  return most;
}

// The product itself, after plan_first or launch_maps.
cudaError_t launch_product(const GroupedArgs &given, int dir, cudaStream_t s) {
  TcMaps m = {};
  GroupedArgs g = given;
  if (dir == GROUPED_WGRAD) {
    const bool wide = g.out_dtype == MOE_ELEM_FP32;
    if (g.vec_out && !expert_map(&m.out, g.out_dtype, g.dw, g, g.K, static_cast<long>(g.N) * g.K, wide ? 32 : 64, 32))
      return cudaErrorInvalidValue;
    HostTrace t("grouped_wgrad", s);
    return launch_tc<GROUPED_WGRAD>(m, g, static_cast<long>(g.E) * ((g.N + 255) / 256) * ((g.K + 255) / 256), s);
  }
  g.most = most_tokens(g, dir);
  const long tokens = (g.rows + g.most - 1L) / g.most + (g.E < g.rows ? g.E : g.rows);
  if (dir == GROUPED_GATED) {
    if (!row_maps(m.b, g.dtype, g.x, g.rows, g.K, g.in_x) || !gated_map(&m.a, g)) return cudaErrorInvalidValue;
    HostTrace t("gated_forward", s);
    return launch_tc<GROUPED_GATED>(m, g, tokens * ((g.N / 2 + 127) / 128), s);
  }
  if (dir == GROUPED_FWD) {
    if (!row_maps(m.b, g.dtype, g.x, g.rows, g.K, g.in_x) || !expert_map(&m.a, g.dtype, g.w, g, g.ld_w, g.ld_e, 64, 128))
      return cudaErrorInvalidValue;
    HostTrace t("grouped_forward", s);
    return launch_tc<GROUPED_FWD>(m, g, tokens * ((g.N + 255) / 256), s);
  }
  if (!row_maps(m.b, g.dtype, g.dy, g.rows, g.N, g.in_y) || !expert_map(&m.a, g.dtype, g.w, g, g.ld_w, g.ld_e, 64, 64))
    return cudaErrorInvalidValue;
  HostTrace t("grouped_dgrad", s);
  return launch_tc<GROUPED_DGRAD>(m, g, tokens * ((g.K + 255) / 256), s);
}

}  // namespace

cudaError_t launch_grouped_order(const GroupedArgs &g, cudaStream_t s) {
  HostTrace t("grouped_order", s);
  grouped_maps_kernel<<<1, 128, 0, s>>>(CUtensorMap(), CUtensorMap(), g);
  return cudaGetLastError();
}

cudaError_t launch_grouped_tc(const GroupedArgs &g, int dir, int num_sms, cudaStream_t s) {
  if (dir != GROUPED_WGRAD && g.rows <= 0) return cudaSuccess;
  cudaError_t e = dir == GROUPED_WGRAD ? launch_maps(g, s) : plan_first(g, dir, s);
  if (e == cudaSuccess && dir == GROUPED_WGRAD && g.zeroed) e = launch_grouped_zero(g, num_sms, s);
  return e == cudaSuccess ? launch_product(g, dir, s) : e;
}

// Programmatic dependent launches.  dgrad needs nothing of the launch in front (the
// maps, or the zeros) and starts with it; wgrad starts when dgrad's blocks all run and
// the maps are written, on the SMs that dgrad does not fill or has left, and ends
// after dgrad.  2043 rows, 8 experts of [512, 768]: 24 us where launches in turn take
// 33; 16384 rows, 32 of [1024, 1024]: 83 and 93; 8192 rows, 8 of [4096, 4096]: 344 and
// 354.  Not wgrad's of the longest products, where 10 us are nothing and pairs that
// start it at different times find less of each other's tiles in L2: 32768 rows, 64 of
// [7168, 2048], 1432 and 1482 us with two draws of the offsets where launches in turn
// take 1441 and 1443.
cudaError_t launch_grouped_tc_pair(GroupedArgs dgrad, GroupedArgs wgrad, int num_sms, cudaStream_t s) {
  dgrad.chained = true;
  wgrad.chained = static_cast<double>(dgrad.rows) * dgrad.N * dgrad.K <= 274877906944.0;
  cudaError_t e = plan_first(dgrad, GROUPED_DGRAD, s);
  if (e == cudaSuccess) e = launch_maps(wgrad, s);
  if (e == cudaSuccess && wgrad.zeroed) e = launch_grouped_zero(wgrad, num_sms, s);
  if (e == cudaSuccess) e = launch_product(dgrad, GROUPED_DGRAD, s);
  if (e == cudaSuccess) e = launch_product(wgrad, GROUPED_WGRAD, s);
  return e;
}

}  // namespace moe
