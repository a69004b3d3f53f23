// Matrix products grouped by expert with ragged sizes: the plan that every
// direction starts with, and the plain tiled kernel that takes any size,
// stride and alignment.
//   y[r] = x[r] w[e]^T,   dx[r] = dy[r] w[e],   dw[e] = sum over e's rows of dy[r]^T x[r]
// Each direction is one matrix product per expert, out[m, n] = sum_k a[m, k] b[n, k],
// whose operands are addressed by two strides; only which index is ragged
// differs (m for y and dx, k for dw).
#include "block.h"
#include "elem.cuh"
#include "gate_act.cuh"
#include "grouped.cuh"
#include "kernels.h"

namespace moe {

namespace {

// ---------------------------------------------------------------- plan
// Block 0: the status word, and the first tile of every expert.  The other
// blocks: zeros for the rows of `out` that belong to no expert.
__global__ void __launch_bounds__(1024) grouped_plan_kernel(const GroupedArgs g, int tile_rows, uint8_t *out,
                                                            long row_bytes, long ld_bytes) {
  pdl_trigger();
  if (blockIdx.x > 0) {
    int lo, hi, lo_last, hi_last;
    group_rows(g, 0, lo, hi);
    group_rows(g, g.E - 1, lo_last, hi_last);
    const long outside = lo + static_cast<long>(g.rows - hi_last);
    for (long i = blockIdx.x - 1; i < outside; i += gridDim.x - 1) {
      const long row = i < lo ? i : hi_last + (i - lo);
      uint8_t *p = out + row * ld_bytes;
      for (long b = threadIdx.x * 2L; b < row_bytes; b += blockDim.x * 2L) *reinterpret_cast<uint16_t *>(p + b) = 0;
    }
    return;
  }
  __shared__ int scratch[256];
  if (tile_rows == 0) {
    const bool bad_offsets = build_tile_table<1024>(g, g.tiles, scratch);
    if (threadIdx.x == 0) *g.status = bad_offsets ? kStatusBounds : 0;
    return;
  }
  __shared__ int warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int run = 0;
  bool bad = false;
  for (int e = threadIdx.x; e < g.E; e += 1024) {
    int lo, hi;
    bad |= !group_rows(g, e, lo, hi);
  }
  const int any = __syncthreads_or(bad);  // bad offsets: no tiles at all
  for (int base = 0; base < g.E; base += 1024) {
    const int e = base + threadIdx.x;
    int n = 0;
    if (e < g.E && !any) {
      int lo, hi;
      group_rows(g, e, lo, hi);
      n = (hi - lo + tile_rows - 1) / tile_rows;
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    if (e < g.E) g.tiles[e] = run + before + inc - n;
    run += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    g.tiles[g.E] = run;
    *g.status = any ? kStatusBounds : 0;
  }
}

// ---------------------------------------------------------------- plain kernel
// 64 x 64 output tiles, 32 of the reduction at a time: loads by element along
// the operand's contiguous index, the next step's in registers while
// mma.sync works on this one's.  It exists for sizes and alignments that TMA
// cannot address, where calls are small.
constexpr int PT = 64, PK = 32, PLD = PK + 8;

template <typename T>
MOE_DEV void mma_16816(float *c, const uint32_t *a, const uint32_t *b);
template <>
MOE_DEV void mma_16816<__nv_bfloat16>(float *c, const uint32_t *a, const uint32_t *b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <>
MOE_DEV void mma_16816<__half>(float *c, const uint32_t *a, const uint32_t *b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

MOE_DEV void ldmatrix4(uint32_t *r, const void *p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}

// One operand tile [PT, PK] of 128 threads: element (i, k) at p + i s_i + k s_k.
struct Side {
  const uint16_t *p;
  long s_i, s_k;
  int ni, nk;  // valid i and k from p on
  MOE_DEV void load(uint16_t *r, int k0) const {
#pragma unroll
    for (int j = 0; j < PT * PK / 128; ++j) {
      const int t = threadIdx.x + j * 128;
      const int i = s_k == 1 ? t / PK : t % PT, k = s_k == 1 ? t % PK : t / PT;
      r[j] = (i < ni && k0 + k < nk) ? p[i * s_i + (k0 + k) * s_k] : static_cast<uint16_t>(0);
    }
  }
  MOE_DEV void put(uint16_t (*sm)[PLD], const uint16_t *r) const {
#pragma unroll
    for (int j = 0; j < PT * PK / 128; ++j) {
      const int t = threadIdx.x + j * 128;
      const int i = s_k == 1 ? t / PK : t % PT, k = s_k == 1 ? t % PK : t / PT;
      sm[i][k] = r[j];
    }
  }
};

// CHAINS: sums over rows are joined in fp32 from chains of this many steps.  The matrix
// instruction truncates what it has added up, always towards zero: over 2^20 rows of one sign
// one chain came out 4e-3 of its size too low.
constexpr int kPlainChain = 2048;

template <typename T, bool CHAINS = false>
MOE_DEV void plain_tile(const Side &a, const Side &b, int nk, float acc[2][4][4]) {
  __shared__ uint16_t sa[PT][PLD], sb[PT][PLD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = (warp & 1) * 32, wn = (warp >> 1) * 32;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][j][k] = 0.f;
  float sum[2][4][4];  // of the chains before this one
  bool more = false;
  uint16_t ra[PT * PK / 128], rb[PT * PK / 128];
  if (nk > 0) {
    a.load(ra, 0);
    b.load(rb, 0);
  }
  for (int k0 = 0; k0 < nk; k0 += PK) {
    __syncthreads();
    a.put(sa, ra);
    b.put(sb, rb);
    __syncthreads();
    if (k0 + PK < nk) {
      a.load(ra, k0 + PK);
      b.load(rb, k0 + PK);
    }
#pragma unroll
    for (int kk = 0; kk < PK; kk += 16) {
      uint32_t fa[2][4], fb[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) ldmatrix4(fa[i], &sa[wm + i * 16 + (lane & 15)][kk + (lane >> 4) * 8]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        ldmatrix4(fb[j], &sb[wn + j * 16 + (lane & 7) + ((lane >> 4) << 3)][kk + ((lane >> 3) & 1) * 8]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_16816<T>(acc[i][j], fa[i], &fb[j >> 1][(j & 1) * 2]);
    }
    const bool last = k0 + PK >= nk;
    if (CHAINS && ((k0 + PK) % kPlainChain == 0 || last) && (more || !last)) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            sum[i][j][k] = more ? sum[i][j][k] + acc[i][j][k] : acc[i][j][k];
            acc[i][j][k] = last ? sum[i][j][k] : 0.f;
          }
      more = true;
    }
  }
}

template <typename T>
MOE_DEV void store_elem(void *out, long at, float v, bool wide, bool add) {
  if (wide) {
    float *p = static_cast<float *>(out) + at;
    *p = add ? *p + v : v;
  } else {
    static_cast<T *>(out)[at] = Elem<T>::from(v);
  }
}

// Accumulator element (i, j, k) of a warp's 32 x 32 part -> row and column.
MOE_DEV void acc_place(int warp, int lane, int i, int j, int k, int &m, int &n) {
  m = (warp & 1) * 32 + i * 16 + (lane >> 2) + (k >> 1) * 8;
  n = (warp >> 1) * 32 + j * 8 + (lane & 3) * 2 + (k & 1);
}

template <typename T, int DIR>
__global__ void __launch_bounds__(128) grouped_plain_kernel(const GroupedArgs g) {
  pdl_wait();  // the plan's tile table, read by ordinary loads: it is written while this kernel may already run
  Side a, b;
  int lo, hi, n0, m0, mn, nn, nk;
  void *out;
  long ldo;
  bool wide, add = false;
  if constexpr (DIR == GROUPED_WGRAD) {
    const int nt = (g.K + PT - 1) / PT, e = blockIdx.y;
    m0 = static_cast<int>(blockIdx.x) / nt * PT;
    n0 = static_cast<int>(blockIdx.x) % nt * PT;
    group_rows(g, e, lo, hi);
    if (lo == hi && (g.accumulate || g.zeroed)) return;
    nk = hi - lo;
    mn = g.N - m0;
    nn = g.K - n0;
    a = Side{static_cast<const uint16_t *>(g.dy) + lo * g.ld_y + m0, 1, g.ld_y, mn, nk};
    b = Side{static_cast<const uint16_t *>(g.x) + lo * g.ld_x + n0, 1, g.ld_x, nn, nk};
    wide = g.out_dtype == MOE_ELEM_FP32;
    add = g.accumulate != 0;
    out = static_cast<uint8_t *>(g.dw) +
          (static_cast<long>(e) * g.N * g.K + static_cast<long>(m0) * g.K + n0) * (wide ? 4 : 2);
    ldo = g.K;
  } else {
    if (static_cast<int>(blockIdx.x) >= g.tiles[g.E]) return;
    const int e = group_of_tile(g.tiles, g.E, blockIdx.x);
    group_rows(g, e, lo, hi);
    m0 = lo + (blockIdx.x - g.tiles[e]) * PT;
    n0 = blockIdx.y * PT;
    mn = hi - m0;
    const uint16_t *w = static_cast<const uint16_t *>(g.w) + static_cast<long>(e) * g.ld_e;
    if constexpr (DIR == GROUPED_FWD) {
      nk = g.K;
      nn = g.N - n0;
      a = Side{static_cast<const uint16_t *>(g.x) + m0 * g.ld_x, g.ld_x, 1, mn, nk};
      b = Side{w + n0 * g.ld_w, g.ld_w, 1, nn, nk};
      wide = g.out_dtype == MOE_ELEM_FP32;
      out = static_cast<uint8_t *>(g.y) + (m0 * g.ld_y + n0) * (wide ? 4 : 2);
      ldo = g.ld_y;
    } else {
      nk = g.N;
      nn = g.K - n0;
      a = Side{static_cast<const uint16_t *>(g.dy) + m0 * g.ld_y, g.ld_y, 1, mn, nk};
      b = Side{w + n0, 1, g.ld_w, nn, nk};
      wide = false;
      out = static_cast<uint8_t *>(g.dx) + (m0 * g.ld_x + n0) * 2;
      ldo = g.ld_x;
    }
  }
  float acc[2][4][4];
  plain_tile<T, DIR == GROUPED_WGRAD>(a, b, nk, acc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        int m, n;
        acc_place(warp, lane, i, j, k, m, n);
        if (m < mn && n < nn) store_elem<T>(out, m * ldo + n, acc[i][j][k], wide, add);
      }
}

// The gated forward: a tile of h from the tiles of both projections.
template <typename T, int ACT>
__global__ void __launch_bounds__(128) gated_plain_kernel(const GroupedArgs g) {
  pdl_wait();  // the plan's tile table
  if (static_cast<int>(blockIdx.x) >= g.tiles[g.E]) return;
  const int e = group_of_tile(g.tiles, g.E, blockIdx.x), half = g.N >> 1;
  int lo, hi;
  group_rows(g, e, lo, hi);
  const int m0 = lo + (blockIdx.x - g.tiles[e]) * PT, n0 = blockIdx.y * PT, mn = hi - m0, nn = half - n0;
  const uint16_t *w = static_cast<const uint16_t *>(g.w) + static_cast<long>(e) * g.ld_e;
  const Side a{static_cast<const uint16_t *>(g.x) + m0 * g.ld_x, g.ld_x, 1, mn, g.K};
  float gate[2][4][4], up[2][4][4];
  plain_tile<T>(a, Side{w + n0 * g.ld_w, g.ld_w, 1, nn, g.K}, g.K, gate);
  plain_tile<T>(a, Side{w + (half + static_cast<long>(n0)) * g.ld_w, g.ld_w, 1, nn, g.K}, g.K, up);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  T *h = static_cast<T *>(g.h) + m0 * g.ld_h + n0, *y = g.y ? static_cast<T *>(g.y) + m0 * g.ld_y + n0 : nullptr;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        int m, n;
        acc_place(warp, lane, i, j, k, m, n);
        if (m < mn && n < nn) {
          h[m * g.ld_h + n] = Elem<T>::from(act_value<ACT>(gate[i][j][k]) * up[i][j][k]);
          if (y) {
            y[m * g.ld_y + n] = Elem<T>::from(gate[i][j][k]);
            y[m * g.ld_y + half + n] = Elem<T>::from(up[i][j][k]);
          }
        }
      }
}

template <typename T>
cudaError_t gated_plain_type(const GroupedArgs &g, cudaStream_t s) {
  const long slots = (g.rows + PT - 1L) / PT + (g.E < g.rows ? g.E : g.rows);
  const dim3 grid(slots, ((g.N >> 1) + PT - 1) / PT);
  switch (g.act) {
    case MOE_ACT_SILU: return launch_early(gated_plain_kernel<T, MOE_ACT_SILU>, grid, 128, s, g);
    case MOE_ACT_GELU: return launch_early(gated_plain_kernel<T, MOE_ACT_GELU>, grid, 128, s, g);
    case MOE_ACT_GELU_TANH: return launch_early(gated_plain_kernel<T, MOE_ACT_GELU_TANH>, grid, 128, s, g);
    default: return launch_early(gated_plain_kernel<T, MOE_ACT_RELU>, grid, 128, s, g);
  }
}

template <typename T>
cudaError_t plain_type(const GroupedArgs &g, int dir, bool planned, cudaStream_t s) {
  const long slots = (g.rows + PT - 1L) / PT + (g.E < g.rows ? g.E : g.rows);
  if (dir == GROUPED_WGRAD) {
    const dim3 grid(((g.N + PT - 1) / PT) * ((g.K + PT - 1) / PT), g.E);
    if (planned) return launch_early(grouped_plain_kernel<T, GROUPED_WGRAD>, grid, 128, s, g);
    grouped_plain_kernel<T, GROUPED_WGRAD><<<grid, 128, 0, s>>>(g);
  } else if (dir == GROUPED_FWD) {
    const dim3 grid(slots, (g.N + PT - 1) / PT);
    if (slots) return launch_early(grouped_plain_kernel<T, GROUPED_FWD>, grid, 128, s, g);
  } else {
    const dim3 grid(slots, (g.K + PT - 1) / PT);
    if (slots) return launch_early(grouped_plain_kernel<T, GROUPED_DGRAD>, grid, 128, s, g);
  }
  return cudaGetLastError();
}

// ---------------------------------------------------------------- few rows
// A generated token: few rows, nearly each with an expert of its own, so the
// work is reading those experts' weights once.  A warp forms FEW_F features of
// up to FEW_R rows of one expert; its lanes split K in 16-byte pieces, FEW_F x
// UNROLL of them in flight each, and join by shuffles in a fixed order.  Block
// (features, row): the first row of every FEW_R rows of an expert does the
// work, the others leave at once.
constexpr int FEW_F = 4, FEW_R = 4, FEW_WARPS = 4;

// GATED: the weights' rows are FEW_F / 2 of the gate and the same of the up projection.
template <bool GATED>
MOE_DEV int few_row(const GroupedArgs &g, int f) {
  return GATED && f >= FEW_F / 2 ? (g.N >> 1) + f - FEW_F / 2 : f;
}
template <bool GATED>
MOE_DEV bool few_has(int f, int nf) {
  return (GATED ? f % (FEW_F / 2) : f) < nf;
}

template <typename T, int R, bool GATED>
MOE_DEV void few_dot(const GroupedArgs &g, const T *x, const T *w, int nf, float acc[R][FEW_F]) {
  const int lane = threadIdx.x & 31, chunks = g.K >> 3;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int f = 0; f < FEW_F; ++f) acc[r][f] = 0.f;
  constexpr int UNROLL = 2;
  for (int c0 = lane; c0 < chunks; c0 += 32 * UNROLL) {
    uint4 q[UNROLL][FEW_F];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
#pragma unroll
      for (int f = 0; f < FEW_F; ++f) {
        q[u][f] = make_uint4(0, 0, 0, 0);
        if (c0 + 32 * u < chunks && few_has<GATED>(f, nf)) q[u][f] = ld_stream(w + few_row<GATED>(g, f) * g.ld_w + (c0 + 32 * u) * 8L);
      }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (c0 + 32 * u >= chunks) break;
      float xv[R][8];
#pragma unroll
      for (int r = 0; r < R; ++r)
        Elem<T>::unpack(__ldg(reinterpret_cast<const uint4 *>(x + r * g.ld_x + (c0 + 32 * u) * 8L)), xv[r]);
#pragma unroll
      for (int f = 0; f < FEW_F; ++f) {
        float wv[8];
        Elem<T>::unpack(q[u][f], wv);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[r][f] = fmaf(xv[r][k], wv[k], acc[r][f]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int f = 0; f < FEW_F; ++f)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][f] += __shfl_xor_sync(0xffffffffu, acc[r][f], o);
}

template <typename T, int R>
MOE_DEV void few_rows(const GroupedArgs &g, int row, int e, int n0, int nf) {
  const int lane = threadIdx.x & 31;
  float acc[R][FEW_F];
  few_dot<T, R, false>(g, static_cast<const T *>(g.x) + row * g.ld_x,
                       static_cast<const T *>(g.w) + e * g.ld_e + n0 * g.ld_w, nf, acc);
  // lane r * FEW_F + f stores element (r, f)
  float v = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int f = 0; f < FEW_F; ++f)
      if (lane == r * FEW_F + f) v = acc[r][f];
  const int r = lane / FEW_F, f = lane % FEW_F;
  if (r < R && f < nf)
    store_elem<T>(g.y, (row + r) * g.ld_y + n0 + f, v, g.out_dtype == MOE_ELEM_FP32, false);
}

template <typename T, int R, int ACT>
MOE_DEV void few_gated_rows(const GroupedArgs &g, int row, int e, int n0, int nf) {
  const int lane = threadIdx.x & 31, half = g.N >> 1;
  float acc[R][FEW_F];
  few_dot<T, R, true>(g, static_cast<const T *>(g.x) + row * g.ld_x,
                      static_cast<const T *>(g.w) + e * g.ld_e + n0 * g.ld_w, nf, acc);
  // lane r * FEW_F / 2 + f stores feature f of row r
  float gate = 0.f, up = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int f = 0; f < FEW_F / 2; ++f)
      if (lane == r * (FEW_F / 2) + f) {
        gate = acc[r][f];
        up = acc[r][f + FEW_F / 2];
      }
  const int r = lane / (FEW_F / 2), f = lane % (FEW_F / 2);
  if (r < R && f < nf) {
    static_cast<T *>(g.h)[(row + r) * g.ld_h + n0 + f] = Elem<T>::from(act_value<ACT>(gate) * up);
    if (g.y) {
      T *y = static_cast<T *>(g.y) + (row + r) * g.ld_y + n0 + f;
      y[0] = Elem<T>::from(gate);
      y[half] = Elem<T>::from(up);
    }
  }
}

// The expert of a row, by the whole block; `lo`, `hi`: its rows (not around the row where
// that belongs to no expert).
MOE_DEV int few_expert(const GroupedArgs &g, int row, int &lo, int &hi) {
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    bool bad = false;
    for (int e = threadIdx.x; e < g.E; e += blockDim.x) bad |= !group_rows(g, e, lo, hi);
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) *g.status = any ? kStatusBounds : 0;
  }
  // experts that end at or before this row = the expert of the row
  int before = 0;
  for (int base = 0; base < g.E; base += blockDim.x) {
    const int e = base + threadIdx.x;
    before += __syncthreads_count(e < g.E && __ldg(g.offsets + e + 1) <= row);
  }
  const int e = before < g.E ? before : g.E - 1;
  group_rows(g, e, lo, hi);
  return e;
}

template <typename T>
__global__ void __launch_bounds__(FEW_WARPS * 32) grouped_few_kernel(const GroupedArgs g) {
  const int row = blockIdx.y;
  int lo, hi;
  const int e = few_expert(g, row, lo, hi);
  const int n0 = (blockIdx.x * FEW_WARPS + (threadIdx.x >> 5)) * FEW_F;
  if (n0 >= g.N) return;
  const int nf = g.N - n0 < FEW_F ? g.N - n0 : FEW_F;
  if (row < lo || row >= hi) {  // a row of no expert
    if (static_cast<int>(threadIdx.x & 31) < nf)
      store_elem<T>(g.y, row * g.ld_y + n0 + (threadIdx.x & 31), 0.f, g.out_dtype == MOE_ELEM_FP32, false);
    return;
  }
  if ((row - lo) % FEW_R) return;
  switch (hi - row) {
    case 1: few_rows<T, 1>(g, row, e, n0, nf); break;
    case 2: few_rows<T, 2>(g, row, e, n0, nf); break;
    case 3: few_rows<T, 3>(g, row, e, n0, nf); break;
    default: few_rows<T, 4>(g, row, e, n0, nf); break;
  }
}

template <typename T, int ACT>
__global__ void __launch_bounds__(FEW_WARPS * 32) gated_few_kernel(const GroupedArgs g) {
  const int row = blockIdx.y, half = g.N >> 1;
  int lo, hi;
  const int e = few_expert(g, row, lo, hi);
  const int n0 = (blockIdx.x * FEW_WARPS + (threadIdx.x >> 5)) * (FEW_F / 2);
  if (n0 >= half) return;
  const int nf = half - n0 < FEW_F / 2 ? half - n0 : FEW_F / 2;
  if (row < lo || row >= hi) {  // a row of no expert
    const int f = threadIdx.x & 31;
    if (f < nf) {
      static_cast<T *>(g.h)[row * g.ld_h + n0 + f] = Elem<T>::from(0.f);
      if (g.y) {
        static_cast<T *>(g.y)[row * g.ld_y + n0 + f] = Elem<T>::from(0.f);
        static_cast<T *>(g.y)[row * g.ld_y + half + n0 + f] = Elem<T>::from(0.f);
      }
    }
    return;
  }
  if ((row - lo) % FEW_R) return;
  switch (hi - row) {
    case 1: few_gated_rows<T, 1, ACT>(g, row, e, n0, nf); break;
    case 2: few_gated_rows<T, 2, ACT>(g, row, e, n0, nf); break;
    case 3: few_gated_rows<T, 3, ACT>(g, row, e, n0, nf); break;
    default: few_gated_rows<T, 4, ACT>(g, row, e, n0, nf); break;
  }
}

template <typename T>
cudaError_t gated_few_type(const GroupedArgs &g, cudaStream_t s) {
  const int per = FEW_WARPS * FEW_F / 2;
  const dim3 grid(((g.N >> 1) + per - 1) / per, g.rows);
  switch (g.act) {
    case MOE_ACT_SILU: gated_few_kernel<T, MOE_ACT_SILU><<<grid, FEW_WARPS * 32, 0, s>>>(g); break;
    case MOE_ACT_GELU: gated_few_kernel<T, MOE_ACT_GELU><<<grid, FEW_WARPS * 32, 0, s>>>(g); break;
    case MOE_ACT_GELU_TANH: gated_few_kernel<T, MOE_ACT_GELU_TANH><<<grid, FEW_WARPS * 32, 0, s>>>(g); break;
    default: gated_few_kernel<T, MOE_ACT_RELU><<<grid, FEW_WARPS * 32, 0, s>>>(g); break;
  }
  return cudaGetLastError();
}

// ---------------------------------------------------------------- zeros
// Pieces of 64 KB of the matrices of the experts without rows (the last of `order`),
// taken in turns.  Whole 16-byte units between a piece's ragged ends.
constexpr long kZeroPiece = 64 << 10;
__global__ void __launch_bounds__(256) grouped_zero_kernel(const GroupedArgs g, long bytes, int pieces) {
  pdl_wait();  // the order
  pdl_trigger();
  const int first = g.order[g.E];
  const long total = static_cast<long>(g.E - first) * pieces;
  for (long u = blockIdx.x; u < total; u += gridDim.x) {
    const long q = u / pieces, e = g.order[first + q];
    const long from = (u - q * pieces) * kZeroPiece;
    const long to = from + kZeroPiece < bytes ? from + kZeroPiece : bytes;
    uint8_t *p = static_cast<uint8_t *>(g.dw) + e * bytes + from;
    const long n = to - from;
    long head = (16 - static_cast<long>(reinterpret_cast<uintptr_t>(p) & 15u)) & 15;
    if (head > n) head = n;
    const long body = (n - head) / 16 * 16;
    for (long b = threadIdx.x * 16L; b < body; b += 256 * 16) st_stream(p + head + b, make_uint4(0, 0, 0, 0));
    // ends: a few elements, 2 bytes at a time
    for (long b = threadIdx.x * 2L; b < head; b += 512) *reinterpret_cast<uint16_t *>(p + b) = 0;
    for (long b = head + body + threadIdx.x * 2L; b < n; b += 512) *reinterpret_cast<uint16_t *>(p + b) = 0;
  }
}

// ---------------------------------------------------------------- padded copies
// Rows at odd strides into rows that TMA can address: a thread per 8 elements.
__global__ void __launch_bounds__(256) grouped_pad_kernel(const GroupedArgs g, const uint16_t *src, long rows, int cols,
                                                          long ld, bool experts, uint16_t *dst, long ld_dst) {
  const int chunks = static_cast<int>(ld_dst >> 3);
  const long total = rows * chunks;
  for (long u = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; u < total;
       u += static_cast<long>(gridDim.x) * blockDim.x) {
    const long row = u / chunks;
    const int c = static_cast<int>(u - row * chunks) * 8;
    const uint16_t *p = src + row * ld + c;
    if (experts) {
      const int e = static_cast<int>(row / g.N);
      int lo, hi;
      group_rows(g, e, lo, hi);
      if (lo == hi) continue;
      p = src + e * g.ld_e + (row - static_cast<long>(e) * g.N) * ld + c;
    }
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = c + 2 * k < cols ? p[2 * k] : 0u, b = c + 2 * k + 1 < cols ? p[2 * k + 1] : 0u;
      w[k] = a | (b << 16);
    }
    *reinterpret_cast<uint4 *>(dst + row * ld_dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

cudaError_t launch_grouped_zero(const GroupedArgs &g, int num_sms, cudaStream_t s) {
  HostTrace t("grouped_zero", s);
  const long bytes = static_cast<long>(g.N) * g.K * elem_bytes(g.out_dtype);
  const int pieces = static_cast<int>((bytes + kZeroPiece - 1) / kZeroPiece);
  // the last wave of many blocks shares the SMs with the data gradient's, launched next (510
  // experts of [448, 3896]: 260 us; with 16 per SM 268, 4 per SM 290)
  const long want = static_cast<long>(g.E) * pieces, most = num_sms * 32L;
  return launch_early(grouped_zero_kernel, static_cast<unsigned>(want < most ? want : most), 256, s, g, bytes, pieces);
}

cudaError_t launch_grouped_pad(const GroupedArgs &g, const void *src, long rows, int cols, long ld, bool experts,
                               void *dst, long ld_dst, cudaStream_t s) {
  HostTrace t("grouped_pad", s);
  const long want = (rows * (ld_dst >> 3) + 255) / 256;
  grouped_pad_kernel<<<static_cast<unsigned>(want < 152 * 32 ? want : 152 * 32), 256, 0, s>>>(
      g, static_cast<const uint16_t *>(src), rows, cols, ld, experts, static_cast<uint16_t *>(dst), ld_dst);
  return cudaGetLastError();
}

cudaError_t launch_gated_few(const GroupedArgs &g, cudaStream_t s) {
  HostTrace t("gated_few", s);
  return g.dtype == MOE_ELEM_BF16 ? gated_few_type<__nv_bfloat16>(g, s) : gated_few_type<__half>(g, s);
}

cudaError_t launch_grouped_few(const GroupedArgs &g, cudaStream_t s) {
  HostTrace t("grouped_few", s);
  const dim3 grid((g.N + FEW_WARPS * FEW_F - 1) / (FEW_WARPS * FEW_F), g.rows);
  if (g.dtype == MOE_ELEM_BF16) grouped_few_kernel<__nv_bfloat16><<<grid, FEW_WARPS * 32, 0, s>>>(g);
  else grouped_few_kernel<__half><<<grid, FEW_WARPS * 32, 0, s>>>(g);
  return cudaGetLastError();
}

cudaError_t launch_grouped_plan(const GroupedArgs &g, int tile_rows, void *out, int out_elem, int out_cols,
                                long ld_out, cudaStream_t s) {
  HostTrace t("grouped_plan", s);
  const long esz = elem_bytes(out_elem);
  const int zero_blocks = out && g.rows > 0 ? (g.rows < 64 ? g.rows : 64) : 0;
  grouped_plan_kernel<<<1 + zero_blocks, 1024, 0, s>>>(g, tile_rows, static_cast<uint8_t *>(out), out_cols * esz,
                                                       ld_out * esz);
  return cudaGetLastError();
}

cudaError_t launch_grouped_plain(const GroupedArgs &g, int dir, bool first, cudaStream_t s) {
  if (first) {
    const bool fwd = dir == GROUPED_FWD;
    const cudaError_t e = launch_grouped_plan(g, PT, fwd ? g.y : (dir == GROUPED_DGRAD ? g.dx : nullptr),
                                              fwd ? g.out_dtype : g.dtype, fwd ? g.N : g.K, fwd ? g.ld_y : g.ld_x, s);
    if (e != cudaSuccess) return e;
  }
  HostTrace t(dir == GROUPED_FWD ? "grouped_fwd_plain" : dir == GROUPED_DGRAD ? "grouped_dgrad_plain" : "grouped_wgrad_plain", s);
  return g.dtype == MOE_ELEM_BF16 ? plain_type<__nv_bfloat16>(g, dir, first, s) : plain_type<__half>(g, dir, first, s);
}

cudaError_t launch_gated_plain(const GroupedArgs &g, cudaStream_t s) {
  if (g.rows == 0) return launch_grouped_plan(g, PT, nullptr, g.dtype, 0, 0, s);
  cudaError_t e = cudaSuccess;
  if (g.y) e = launch_grouped_plan(g, PT, g.y, g.dtype, g.N, g.ld_y, s);
  if (e == cudaSuccess) e = launch_grouped_plan(g, PT, g.h, g.dtype, g.N >> 1, g.ld_h, s);
  if (e != cudaSuccess) return e;
  HostTrace t("gated_plain", s);
  return g.dtype == MOE_ELEM_BF16 ? gated_plain_type<__nv_bfloat16>(g, s) : gated_plain_type<__half>(g, s);
}

}  // namespace moe
