// The products behind the loss over a vocabulary on CTA pairs (tcgen05, cta_group::2):
//
//   LOSS  logits z = xs w^T of 256 rows x 256 vocabulary entries; of a row's logits but its
//         label's the maximum and the sum of exponentials leave, the logits do not
//   DZ    the same logits again, out as dz = coef_p exp(z - lse) (the label's: its own
//         value) in 16 bits, one piece of the vocabulary at a time
//   DX    sum += dz w over a piece            A = dz K-major,  B = w read MN-major
//   DW    dw = dz^T xs                        A and B read MN-major
//
// With the rows on the instruction's M side a thread of the epilogue owns one
// row: maximum and sum stay in its registers, without a shuffle.  Rows are
// dense here (those that do not count were left out by the copy), so tiles are
// whole; what a tile has past the last row or column is computed on zeros that TMA
// fills in and not stored.
//
// Bound by the tensor cores from some 512 rows on, by reading w below.
//
// Roles per CTA (320 threads) as in the grouped products: TMA producer, MMA issuer
// (leader CTA), eight epilogue warps; three 64 KB stages of two blocks of 64
// reduction steps; two accumulators of 256 TMEM columns.  Persistent over pairs.
// Tiles are taken in bands of a few row tiles, so that a band's rows stay in L2
// while the other operand streams by.  Every wait is bounded (mbar_wait).
#include <type_traits>

#include "elem.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

#include "block.h"

namespace moe {

namespace {

constexpr int kBlockBytes = 32768;  // 64 reduction steps: 16 KB of A, 16 KB of B
constexpr int kThreads = 320;
constexpr int kEpilogueWarps = 8;
constexpr int kStaging = 4096;      // per epilogue warp
constexpr int kBlocks = 2, kStages = 3;
constexpr int kStageBytes = kBlocks * kBlockBytes;
constexpr size_t kSmem = 1024 + kStages * kStageBytes + kEpilogueWarps * kStaging + (2 * kStages + 5) * 8 + 16;
static_assert(kSmem <= 232448, "shared memory");
// Row tiles of a band (16384 rows, 131072 x 4096, logits of the forward: 10.69 ms with 4,
// 10.04 with 8, 9.99 with 12, 9.92 with 16, 10.0 with 32; the backward's products are best
// with 8 to 12).
template <int MODE>
constexpr int kBand = MODE == VOCAB_LOSS ? 16 : 8;
constexpr float kLog2e = 1.44269504088896340736f;
// Up to here a logit times log2 e stays in fp32.
constexpr float kMostBase = 2.3e38f;

struct VocabMaps {
  CUtensorMap a, b, out;
};

MOE_DEV void tma_store_2d(const CUtensorMap *map, const void *src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
MOE_DEV void tma_add_2d(const CUtensorMap *map, const void *src, int c0, int c1) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
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

// kind::f16, fp32 accumulation, M = 256 over the pair: operand format (1 bf16, 0 fp16) at
// [7,10) and [10,13), MN-major A / B at bits 15 / 16, N >> 3 at [17,23).
template <int MODE>
MOE_DEV uint32_t vocab_idesc(int dtype, int n) {
  const uint32_t f = dtype == MOE_ELEM_BF16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | (MODE == VOCAB_DW ? 1u << 15 : 0u) |
         (MODE == VOCAB_DX || MODE == VOCAB_DW ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (16u << 24);
}

MOE_DEV void tmem_ld16_async(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 2^x in the hardware's approximation (2 ulp), 0 below the normal range.
MOE_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// How many reduction steps one accumulator takes.  An accumulator truncates at every
// instruction, always towards zero: a chain of 448 of them (d = 7168) left logits 1.3e-5 too
// low, all alike, which lse and the loss inherit, and one of 16384 a dw of terms of one sign over
// 262144 rows 4.3e-4 of its size.  LOSS is joined from chains of kChain steps in fp32, and so
// is dw (CHAINS) of more rows than that in fp32 (2.2e-7, whatever the rows), or than kChain16
// in 16 bits (6.7e-5).  dz and dx are rounded to 16 bits, which is more than the chains of a
// width or of a piece of the vocabulary lose.
constexpr int kChain = 2048, kChain16 = 65536;
template <int MODE, bool WIDE, bool CHAINS>
MOE_DEV int chain_of(int klen) {
  return MODE == VOCAB_LOSS || (CHAINS && WIDE) ? kChain : CHAINS ? kChain16 : (klen > 0 ? klen : 1);
}

struct VocabTile {
  int m0, n0;       // first row and column of the product
  int n;            // columns: 256, or 128 at the end of an MN-major B
  int k0, klen;     // reduction
  int split;
};

// LOSS, DZ: rows x vocabulary of the piece; DX: rows x d, the piece's reduction in
// `splits` parts; DW: vocabulary of the piece x d.
template <int MODE>
struct VocabTiles {
  int nm, nn, cols, splits, k, per, total;
  MOE_DEV VocabTiles(const VocabArgs &a, int count) {
    nm = ((MODE == VOCAB_DW ? a.wp : count) + 255) >> 8;
    cols = MODE == VOCAB_LOSS || MODE == VOCAB_DZ ? a.wp : a.d;
    nn = (cols + 255) >> 8;
    splits = MODE == VOCAB_DX ? a.splits : 1;
    k = MODE == VOCAB_DX ? a.wp : MODE == VOCAB_DW ? count : a.d;
    per = ((k + 127) / 128 + splits - 1) / splits * 128;
    total = nm * nn * splits;
  }
  MOE_DEV VocabTile at(int u) const {
    VocabTile t;
    const int plane = nm * nn;
    t.split = u / plane;
    u -= t.split * plane;
    constexpr int tall = kBand<MODE>;
    const int band = u / (tall * nn), in = u - band * tall * nn;
    const int high = nm - band * tall < tall ? nm - band * tall : tall;
    t.m0 = (band * tall + in % high) * 256;
    t.n0 = in / high * 256;
    t.n = (MODE == VOCAB_DX || MODE == VOCAB_DW) && cols - t.n0 <= 128 ? 128 : 256;
    t.k0 = t.split * per;
    t.klen = k - t.k0 < per ? k - t.k0 : per;
    if (t.klen < 0) t.klen = 0;
    return t;
  }
};

// A piece of 32 rows x 128 bytes (lane = row) into 128-byte-swizzled shared memory, from
// where TMA takes it.
MOE_DEV void stage_rows(const uint32_t *w, uint8_t *buf, int lane) {
  if (lane == 0) bulk_wait_read<0>();  // the last piece has left the buffer
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4 *>(buf + lane * 128 + ((j ^ (lane & 7)) * 16)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  fence_proxy_async_smem();
  __syncwarp();
}

// The same piece element by element, for matrices whose rows are no whole 16-byte
// pieces: each store takes neighbouring columns of one row.  (In words of 4 bytes, with
// the odd ends apart: 74 us where this is 49, 515 rows and 50001 x 321.)
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

// T: the operands' type; WIDE: fp32 dw; CHAINS: dw from several accumulators.
template <int MODE, typename T, bool WIDE, bool CHAINS>
__global__ void __launch_bounds__(kThreads, 1) vocab_tc_kernel(const __grid_constant__ VocabMaps maps, const VocabArgs g) {
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
  const bool turns = MODE == VOCAB_DZ || (MODE == VOCAB_LOSS && g.d <= kChain);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * (turns ? kEpilogueWarps / 2 : kEpilogueWarps));  // epilogue warps of both CTAs
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
  pdl_wait();  // all that the launches in front have written, the rows that count among it
  pdl_trigger();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int count = *reinterpret_cast<const volatile int *>(g.count);
  const VocabTiles<MODE> tiles(g, count);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      fence_proxy_async_global();  // copies and dz were written by ordinary stores and by TMA
      int stage = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = pair; u < tiles.total && ok && !*abort_flag; u += pairs) {
        const VocabTile t = tiles.at(u);
        const int ar = t.m0 + static_cast<int>(rank) * 128, br = t.n0 + static_cast<int>(rank) * (t.n >> 1);
        const uint32_t bytes = t.n == 256 ? 32768u : 24576u;  // of a block, per CTA
        for (int kb = 0; kb < t.klen; kb += 64 * kBlocks) {
          if (!mbar_wait(&empty[stage], ph ^ 1u, abort_flag, g.status)) {
            ok = false;
            break;
          }
          const int blocks = t.klen - kb > 64 ? kBlocks : 1;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2u * blocks * bytes);
          const uint32_t bar = peer_smem(smem_u32(&full[stage]), 0);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            if (b >= blocks) break;
            uint8_t *sa = smem + stage * kStageBytes + b * kBlockBytes, *sb = sa + 16384;
            const int k = t.k0 + kb + 64 * b;
            if constexpr (MODE == VOCAB_DW) {
              tma_load_2d_pair(&maps.a, bar, sa, ar, k);
              tma_load_2d_pair(&maps.a, bar, sa + 8192, ar + 64, k);
            } else {
              tma_load_2d_pair(&maps.a, bar, sa, k, ar);
            }
            if constexpr (MODE == VOCAB_DX || MODE == VOCAB_DW) {
              const int kr = MODE == VOCAB_DX ? g.v0 + k : k;
              tma_load_2d_pair(&maps.b, bar, sb, br, kr);
              if (t.n == 256) tma_load_2d_pair(&maps.b, bar, sb + 8192, br + 64, kr);
            } else {
              tma_load_2d_pair(&maps.b, bar, sb, k, g.v0 + br);
            }
          }
          if (++stage == kStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (pair leader)
    if (leader && lane == 0) {
      int stage = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int u = pair; u < tiles.total && ok; u += pairs) {
        const VocabTile t = tiles.at(u);
        const uint32_t idesc = vocab_idesc<MODE>(g.dtype, t.n);
        for (int from = 0, chain = chain_of<MODE, WIDE, CHAINS>(t.klen); from < t.klen && ok; from += chain) {
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
                const uint64_t ad = MODE == VOCAB_DW ? mn_desc(sa + 2048 * (k & 3)) : sw128_desc(sa + 32 * (k & 3));
                const uint64_t bd = MODE == VOCAB_DX || MODE == VOCAB_DW ? mn_desc(sb + 2048 * (k & 3))
                                                                        : sw128_desc(sb + 32 * (k & 3));
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
    // Two groups of four warps.  Where a tile is one accumulator (LOSS of rows up to kChain,
    // DZ) they take tiles in turns, so that one's exponentials run beside the other's
    // loads; else each takes half of the columns.
    const int q = warp & 3, group = (warp - 2) >> 2;
    uint8_t *buf = staging + (warp - 2) * kStaging;
    uint32_t seq = 0;  // accumulators that the pair has taken
    bool lost = false;
    for (int u = pair, i = 0; u < tiles.total && !lost; u += pairs, ++i) {
      if (turns && (i & 1) != group) {
        ++seq;
        continue;
      }
      const VocabTile t = tiles.at(u);
      const int row0 = t.m0 + static_cast<int>(rank) * 128 + q * 32, row = row0 + lane;
      const int col0 = t.n0 + group * 128;
      const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
      uint32_t tb = lanes + (seq & 1) * 256 + group * 128;
      if (t.klen > 0) {
        if (!mbar_wait(&tfull[seq & 1], seq >> 1 & 1, abort_flag, g.status)) break;
        tc_fence_after();
      }
      // one arrival per warp, without an order of its own at cluster scope: one per thread that
      // had it took the other CTA's warps 1600 cycles a tile (5 rows, 131072 x 4096: the
      // weight gradient 268 us, 182 so)
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(&tempty[seq & 1]);
          else mbar_arrive_remote_tmem(peer_smem(smem_u32(&tempty[seq & 1]), 0));
        }
      };
      if constexpr (MODE == VOCAB_LOSS) {
        // d >= 1: klen > 0.  128 logits in registers at a time: the chains' sums meet there.
        const int label = g.label[row] - g.v0;  // rows are padded to whole tiles
        for (int part = turns ? 0 : group; part < (turns ? 2 : group + 1); ++part) {
          float z[128];
          uint32_t *r = reinterpret_cast<uint32_t *>(z);
          tb = lanes + (seq & 1) * 256 + part * 128;
#pragma unroll
          for (int j = 0; j < 128; j += 32) tmem_ld32_async(tb + j, r + j);
          tmem_ld_wait();
          reg_fence<128>(r);
          if (!turns || part == 1) release();
          for (int from = kChain; from < t.klen; from += kChain) {
            ++seq;
            if (!mbar_wait(&tfull[seq & 1], seq >> 1 & 1, abort_flag, g.status)) {
              lost = true;
              break;
            }
            tc_fence_after();
            tb = lanes + (seq & 1) * 256 + part * 128;
#pragma unroll
            for (int j = 0; j < 128; j += 16) {
              uint32_t more[16];
              tmem_ld16_async(tb + j, more);
              tmem_ld_wait();
              reg_fence<16>(more);
#pragma unroll
              for (int i = 0; i < 16; ++i) z[j + i] += __uint_as_float(more[i]);
            }
            release();
          }
          if (lost) break;
          const int first = t.n0 + part * 128, hit = label - first;
          const int left = g.wp - first;  // columns that exist
          if (left < 128) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i >= left) z[i] = -__int_as_float(0x7f800000);
          }
          if (__any_sync(0xffffffffu, hit >= 0 && hit < 128)) {  // the label's logit is formed apart
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (hit == i) z[i] = -__int_as_float(0x7f800000);
          }
          float m0 = z[0], m1 = z[1];
#pragma unroll
          for (int i = 2; i < 128; i += 2) {
            m0 = fmaxf(m0, z[i]);
            m1 = fmaxf(m1, z[i + 1]);
          }
          const float m = fmaxf(m0, m1);
          // a maximum that is not finite: exponentials from zero, as the join expects
          const float base = fabsf(m) <= kMostBase ? m * kLog2e : 0.f;
          if (fabsf(m) > kMostBase && fabsf(m) <= 3.402823466e38f) {  // m log2 e is not: from m by subtraction
#pragma unroll
            for (int i = 0; i < 128; ++i) z[i] -= m;
          }
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 128; ++i) s[i & 3] += ex2(fmaf(z[i], kLog2e, -base));
          if (row < count)
            g.part[static_cast<long>(row) * g.parts + (t.n0 >> 7) + part] = make_float2(m, (s[0] + s[1]) + (s[2] + s[3]));
        }
      } else if constexpr (MODE == VOCAB_DZ) {
        // out through the staging by plain stores: nothing to wait for between pieces
        const float cp = g.coef_p[row], own = g.hit[row];
        float base = g.base[row], less = 0.f;
        if (fabsf(base) > 3.402823466e38f && row < count) {  // lse log2 e: lse itself may be finite
          const float l = g.lse_in[g.row[row]];
          if (fabsf(l) <= 3.402823466e38f) {
            less = l;
            base = 0.f;
          }
        }
        const int label = g.label[row] - (g.v0 + t.n0);
        const gemm_detail::OutView out = gemm_detail::out_view(g.dz, g.width, (g.rows + 127L) / 128 * 128, 2);
#pragma unroll 1
        for (int j = 0; j < 256; j += 64) {
          uint32_t r[64];
          tb = lanes + (seq & 1) * 256 + j;
          tmem_ld32_async(tb, r);
          tmem_ld32_async(tb + 32, r + 32);
          tmem_ld_wait();
          reg_fence<64>(r);
          if (j == 192) release();
          if (t.n0 + j >= g.wp) continue;
          float *z = reinterpret_cast<float *>(r);
          if (less != 0.f) {
#pragma unroll
            for (int i = 0; i < 64; ++i) z[i] -= less;
          }
          // no coefficient, no term: what z holds there does not matter
#pragma unroll
          for (int i = 0; i < 64; ++i) z[i] = cp == 0.f ? 0.f : cp * ex2(fmaf(z[i], kLog2e, -base));
          const int hit = label - j;
          if (__any_sync(0xffffffffu, hit >= 0 && hit < 64)) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (hit == i) z[i] = own;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = Elem<T>::pack2(z[32 * h + 2 * i], z[32 * h + 2 * i + 1]);
            gemm_detail::Stager(buf + h * 2048).put(out, w, t.n0 + j + 32 * h, row0, lane);
          }
        }
      } else if constexpr (MODE == VOCAB_DX) {
#pragma unroll 1
        for (int j = 0; j < 128; j += 32) {
          uint32_t r[32];
          if (group * 128 >= t.n) {  // the narrow tile's columns are the first group's
            if (t.klen > 0) release();
            break;
          }
          if (t.klen > 0) {
            tmem_ld32_async(tb + j, r);
            tmem_ld_wait();
            reg_fence<32>(r);
            if (j == 96) release();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0;
          }
          if (col0 + j >= g.d || row0 >= count || (t.klen == 0 && g.v0 > 0)) continue;
          stage_rows(r, buf, lane);
          if (lane == 0) {
            if (g.v0 > 0) tma_add_3d(&maps.out, buf, col0 + j, row0, t.split);
            else tma_store_3d(&maps.out, buf, col0 + j, row0, t.split);
            bulk_commit();
          }
        }
      } else {
        constexpr int STEP = WIDE ? 32 : 64;  // columns of a 128-byte piece
        if (CHAINS && t.klen > chain_of<MODE, WIDE, CHAINS>(t.klen)) {
          // The chains' sums meet in registers, as in LOSS, and go back to the last one's columns:
          // kept in registers up to the stores they spilled.  (8192 rows, 131072 x 4096: 10.5 ms,
          // 10.3 as one chain; added up in dw by TMA 10.85, and 274 us instead of 146 for 9000 rows
          // and 5001 x 321, whose elements leave one by one.)
          const bool mine = group * 128 < t.n;  // the narrow tile's columns are the first group's
          float z[128];
#pragma unroll
          for (int i = 0; i < 128; ++i) z[i] = 0.f;
          for (int from = 0, chain = chain_of<MODE, WIDE, CHAINS>(t.klen); from < t.klen; from += chain) {
            if (from > 0) {
              release();
              ++seq;
              if (!mbar_wait(&tfull[seq & 1], seq >> 1 & 1, abort_flag, g.status)) {
                lost = true;
                break;
              }
              tc_fence_after();
              tb = lanes + (seq & 1) * 256 + group * 128;
            }
            if (!mine) continue;
#pragma unroll
            for (int j = 0; j < 128; j += 16) {
              uint32_t more[16];
              tmem_ld16_async(tb + j, more);
              tmem_ld_wait();
              reg_fence<16>(more);
#pragma unroll
              for (int i = 0; i < 16; ++i) z[j + i] += __uint_as_float(more[i]);
            }
          }
          if (lost) break;
          if (mine) {
#pragma unroll
            for (int j = 0; j < 128; j += 32) tmem_st32(tb + j, reinterpret_cast<const uint32_t *>(z) + j);
            tmem_st_wait();
          }
        }
        const float scale = *reinterpret_cast<const volatile float *>(g.scale);
#pragma unroll 1
        for (int j = 0; j < 128; j += STEP) {
          uint32_t r[STEP], w[32];
          if (group * 128 >= t.n) {
            if (t.klen > 0) release();
            break;
          }
          if (t.klen > 0) {
            tmem_ld32_async(tb + j, r);
            if (!WIDE) tmem_ld32_async(tb + j + 32, r + STEP - 32);
            tmem_ld_wait();
            reg_fence<STEP>(r);
            if (j + STEP == 128) release();
          } else {
#pragma unroll
            for (int i = 0; i < STEP; ++i) r[i] = 0;
          }
          if (row0 >= g.wp || col0 + j >= g.d || (t.klen == 0 && g.accumulate)) continue;
          float *v = reinterpret_cast<float *>(r);
          if (t.klen > 0)
#pragma unroll
            for (int i = 0; i < STEP; ++i) v[i] *= scale;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if constexpr (WIDE) w[i] = r[i];
            else w[i] = Elem<T>::pack2(v[2 * i], v[2 * i + 1]);
          if (g.vec_dw) {
            stage_rows(w, buf, lane);
            if (lane == 0) {
              if (WIDE && g.accumulate) tma_add_2d(&maps.out, buf, col0 + j, g.v0 + row0);
              else tma_store_2d(&maps.out, buf, col0 + j, g.v0 + row0);
              bulk_commit();
            }
          } else {
            using O = typename std::conditional<WIDE, float, T>::type;
            put_elements<O>(w, buf, static_cast<O *>(g.dw) + static_cast<long>(g.v0 + row0) * g.d + col0 + j, g.d,
                            g.wp - row0, g.d - col0 - j, g.accumulate != 0, lane);
          }
        }
      }
      if (t.klen > 0) ++seq;
    }
    if ((MODE == VOCAB_DX || MODE == VOCAB_DW) && lane == 0) bulk_wait<0>();
  }

  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int MODE, typename T, bool WIDE, bool CHAINS>
int vocab_clusters_query() {
  const auto kernel = vocab_tc_kernel<MODE, T, WIDE, CHAINS>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) != cudaSuccess)
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

template <int MODE, typename T, bool WIDE, bool CHAINS>
cudaError_t launch_kernel(const VocabMaps &maps, const VocabArgs &g, long units, cudaStream_t s) {
  static int memo[64] = {};
  const int most = per_device_memo(memo, vocab_clusters_query<MODE, T, WIDE, CHAINS>);
  if (most <= 0) return cudaErrorInvalidConfiguration;
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
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, vocab_tc_kernel<MODE, T, WIDE, CHAINS>, maps, g);
}

// CHAINS costs registers, and time where there is one chain: 515 rows, 50001 x 321 with dx 169
// us, 152 without.
template <int MODE, typename T, bool WIDE>
cudaError_t launch_one(const VocabMaps &maps, const VocabArgs &g, long units, cudaStream_t s) {
  if constexpr (MODE == VOCAB_DW) {
    if (g.rows > (WIDE ? kChain : kChain16)) return launch_kernel<MODE, T, WIDE, true>(maps, g, units, s);
  }
  return launch_kernel<MODE, T, WIDE, false>(maps, g, units, s);
}

template <int MODE>
cudaError_t launch_mode(const VocabMaps &m, const VocabArgs &g, long units, cudaStream_t s) {
  const bool bf = g.dtype == MOE_ELEM_BF16;
  if constexpr (MODE == VOCAB_DW) {
    if (g.grad_dtype == MOE_ELEM_FP32)
      return bf ? launch_one<MODE, __nv_bfloat16, true>(m, g, units, s) : launch_one<MODE, __half, true>(m, g, units, s);
  }
  return bf ? launch_one<MODE, __nv_bfloat16, false>(m, g, units, s) : launch_one<MODE, __half, false>(m, g, units, s);
}

bool map_2d(CUtensorMap *m, int elem, const void *p, long cols, long rows, long ld, uint32_t box_cols, uint32_t box_rows) {
  const uint64_t e = elem_bytes(elem);
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows > 0 ? rows : 1)};
  const uint64_t strides[1] = {static_cast<uint64_t>(ld) * e};
  const uint32_t box[2] = {box_cols, box_rows};
  return host_encode_map(m, elem, p, 2, dims, strides, box);
}

}  // namespace

cudaError_t launch_vocab_tc(const VocabArgs &g, int mode, cudaStream_t s) {
  VocabMaps m = {};
  const void *w = g.pad_w ? g.ws_w : g.w;
  const long ld_w = g.pad_w ? g.ld_ws_w : g.ld_w;
  const long high = (g.rows + 127L) / 128 * 128;  // rows of the workspace's operands
  const long rt = (g.rows + 255L) / 256, vt = (g.wp + 255L) / 256, dt = (g.d + 255L) / 256;
  if (mode == VOCAB_LOSS || mode == VOCAB_DZ) {
    if (!map_2d(&m.a, g.dtype, g.xs, g.d, high, g.ld_xs, 64, 128) || !map_2d(&m.b, g.dtype, w, g.d, g.V, ld_w, 64, 128))
      return cudaErrorInvalidValue;
    if (mode == VOCAB_LOSS) {
      HostTrace t("vocab_logits", s);
      return launch_mode<VOCAB_LOSS>(m, g, rt * vt, s);
    }
    HostTrace t("vocab_dlogits", s);
    return launch_mode<VOCAB_DZ>(m, g, rt * vt, s);
  }
  if (mode == VOCAB_DX) {
    const uint64_t dims[3] = {static_cast<uint64_t>(g.ld_sum), static_cast<uint64_t>(g.rows), static_cast<uint64_t>(g.splits)};
    const uint64_t strides[2] = {static_cast<uint64_t>(g.ld_sum) * 4, static_cast<uint64_t>(g.ld_sum) * 4 * g.rows};
    const uint32_t box[3] = {32, 32, 1};
    if (!map_2d(&m.a, g.dtype, g.dz, g.wp, high, g.width, 64, 128) ||
        !map_2d(&m.b, g.dtype, w, g.d, g.V, ld_w, 64, 64) || !host_encode_map(&m.out, MOE_ELEM_FP32, g.sum, 3, dims, strides, box))
      return cudaErrorInvalidValue;
    HostTrace t("vocab_dgrad", s);
    return launch_mode<VOCAB_DX>(m, g, rt * dt * g.splits, s);
  }
  const bool wide = g.grad_dtype == MOE_ELEM_FP32;
  if (!map_2d(&m.a, g.dtype, g.dz, g.wp, high, g.width, 64, 64) || !map_2d(&m.b, g.dtype, g.xs, g.d, high, g.ld_xs, 64, 64))
    return cudaErrorInvalidValue;
  if (g.vec_dw && !map_2d(&m.out, g.grad_dtype, g.dw, g.d, g.V, g.d, wide ? 32 : 64, 32)) return cudaErrorInvalidValue;
  HostTrace t("vocab_wgrad", s);
  return launch_mode<VOCAB_DW>(m, g, vt * dt, s);
}

}  // namespace moe
