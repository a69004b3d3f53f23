// The norms around a block, fused with its gate and the residual:
//   n = w_post f / rms(f),  z = alpha x + g n,  h = w_pre z / rms(z),
// and their backward.  With r = 1 / rms and u = r v, du pulls back to
//   dv = r du - v r^3 <du, v> / d,
// so with t = dz + r_pre (w_pre dh) - z r_pre^3 <w_pre dh, z> / d (the gradient
// that reaches z from both sides)
//   dx = alpha t,   dn = g t,   df = r_post (w_post dn) - f r_post^3 <w_post dn, f> / d,
//   dw_pre = sum_rows dh z r_pre,   dw_post = sum_rows dn f r_post,   dg = t n.
// <w_post dn, f> needs t, and t needs <w_pre dh, z>.  Expanding t makes it one
// round of sums over the row:
//   <t, q> = <dz, q> + r_pre <w_pre dh, q> - c <z, q>,  q = w_post g f,
// so the row is read once and a block waits for one reduction per row.
//
// HBM bound: forward 4 elements moved per column (f, x in; z, h out), backward 6
// (dz, dh, z, f in; dx, df out).
#include "gemm_common.cuh"
#include "kernels.h"
#include "norm.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- forward
// Chunks of one row of a tensor (NULL: zeros).
template <typename T, int VEC, int NCH>
MOE_DEV void load_row(Chunk<T, VEC> *q, const void *base, long row, long ld, int d, int tid, int tpr) {
  const T *p = static_cast<const T *>(base) + row * ld;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (tid + i * tpr) * VEC;
    if (base && c < d) q[i].load(p + c);
    else q[i].clear();
  }
}

// A row stays in the registers of its threads (NCH chunks of VEC columns each)
// from the loads to the stores.  The blocks are persistent, and the next row's
// loads are issued before this row's sums: the reductions' waits would
// otherwise leave the memory idle.
template <typename T, int VEC, int NCH, bool WARP, int THREADS, int MINB>
__global__ void __launch_bounds__(THREADS, MINB) norm_fwd_kernel(const NormArgs a) {
  __shared__ float red[2][1][kMaxWarps];
  const int tpr = WARP ? 32 : blockDim.x;
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int rpb = WARP ? (blockDim.x >> 5) : 1;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const long step = static_cast<long>(gridDim.x) * rpb;
  int turn = 0;
  long row = static_cast<long>(blockIdx.x) * rpb + (WARP ? (threadIdx.x >> 5) : 0);
  if (row >= a.rows) return;
  Chunk<T, VEC> xn[NCH], fn[NCH];
  load_row<T, VEC, NCH>(xn, a.x, row, a.ld_x, a.d, tid, tpr);
  load_row<T, VEC, NCH>(fn, a.f, row, a.ld_f, a.d, tid, tpr);
  for (; row < a.rows; row += step) {
    Chunk<T, VEC> xq[NCH], fq[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      xq[i] = xn[i];
      fq[i] = fn[i];
    }
    if (row + step < a.rows) {
      load_row<T, VEC, NCH>(xn, a.x, row + step, a.ld_x, a.d, tid, tpr);
      load_row<T, VEC, NCH>(fn, a.f, row + step, a.ld_f, a.d, tid, tpr);
    }
    float r = 1.f;
    if (a.flags & MOE_NORM_POST) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        float v[VEC];
        fq[i].get(v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) ss[0] = fmaf(v[k], v[k], ss[0]);
      }
      row_sum<WARP, 1>(ss, red, turn);
      r = rsqrtf(ss[0] * inv_d + a.eps);
      if (tid == 0 && a.r_post) a.r_post[row] = r;
    }
    const float rg = row_gate_of<T>(a, row);
    float z[NCH][VEC];
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (tid + i * tpr) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) z[i][k] = 0.f;
      if (c < a.d) {
        xq[i].get(z[i]);
#pragma unroll
        for (int k = 0; k < VEC; ++k) z[i][k] *= a.alpha;
        if (a.f) {
          float v[VEC], w[VEC], g[VEC];
          fq[i].get(v);
          weight_chunk<T, VEC>(a.w_post, c, w);
          gate_chunk<T, VEC>(a, row, c, rg, g);
#pragma unroll
          for (int k = 0; k < VEC; ++k) z[i][k] = fmaf(g[k], v[k] * r * w[k], z[i][k]);
        }
        if (a.z) Chunk<T, VEC>::store(static_cast<T *>(a.z) + row * a.ld_z + c, z[i]);
#pragma unroll
        for (int k = 0; k < VEC; ++k) ss[0] = fmaf(z[i][k], z[i][k], ss[0]);
      }
    }
    if (a.flags & MOE_NORM_PRE) {
      row_sum<WARP, 1>(ss, red, turn);
      r = rsqrtf(ss[0] * inv_d + a.eps);
      if (tid == 0 && a.r_pre) a.r_pre[row] = r;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int c = (tid + i * tpr) * VEC;
        if (c < a.d) {
          float w[VEC];
          weight_chunk<T, VEC>(a.w_pre, c, w);
#pragma unroll
          for (int k = 0; k < VEC; ++k) z[i][k] *= r * w[k];
          Chunk<T, VEC>::store(static_cast<T *>(a.h) + row * a.ld_h + c, z[i]);
        }
      }
    }
  }
}

// Rows that do not fit the registers of a block: each pass reads the row again
// (from L1 / L2).
template <typename T>
__global__ void __launch_bounds__(1024) norm_fwd_long_kernel(const NormArgs a) {
  __shared__ float red[2][1][kMaxWarps];
  const float inv_d = 1.f / static_cast<float>(a.d);
  int turn = 0;
  for (long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T *xr = static_cast<const T *>(a.x) + row * a.ld_x;
    const T *fr = a.f ? static_cast<const T *>(a.f) + row * a.ld_f : nullptr;
    float r = 1.f, ss[1] = {0.f};
    if (a.flags & MOE_NORM_POST) {
      for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        const float v = Elem<T>::to(fr[c]);
        ss[0] = fmaf(v, v, ss[0]);
      }
      row_sum<false, 1>(ss, red, turn);
      r = rsqrtf(ss[0] * inv_d + a.eps);
      if (threadIdx.x == 0 && a.r_post) a.r_post[row] = r;
    }
    const float rg = row_gate_of<T>(a, row);
    auto z_at = [&](int c) {
      float z = a.alpha * Elem<T>::to(xr[c]);
      if (fr) {
        float w, g;
        weight_chunk<T, 1>(a.w_post, c, &w);
        gate_chunk<T, 1>(a, row, c, rg, &g);
        z = fmaf(g, Elem<T>::to(fr[c]) * r * w, z);
      }
      return z;
    };
    ss[0] = 0.f;
    if (a.flags & MOE_NORM_PRE) {
      for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
        const float z = z_at(c);
        ss[0] = fmaf(z, z, ss[0]);
      }
      row_sum<false, 1>(ss, red, turn);
    }
    const float rp = rsqrtf(ss[0] * inv_d + a.eps);
    if ((a.flags & MOE_NORM_PRE) && threadIdx.x == 0 && a.r_pre) a.r_pre[row] = rp;
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
      const float z = z_at(c);   // before the stores: z may be x's or f's buffer
      if (a.z) static_cast<T *>(a.z)[row * a.ld_z + c] = Elem<T>::from(z);
      if (a.flags & MOE_NORM_PRE) {
        float w;
        weight_chunk<T, 1>(a.w_pre, c, &w);
        static_cast<T *>(a.h)[row * a.ld_h + c] = Elem<T>::from(z * (rp * w));
      }
    }
  }
}

// ---------------------------------------------------------------- backward
// Rows in registers, the next row's loads in flight (as the forward).
template <typename T, int VEC, int NCH, bool WARP, int THREADS, int MINB>
__global__ void __launch_bounds__(THREADS, MINB) norm_bwd_kernel(const NormArgs a) {
  pdl_trigger();
  __shared__ float red[2][4][kMaxWarps];
  const int tpr = WARP ? 32 : blockDim.x;
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int rpb = WARP ? (blockDim.x >> 5) : 1;
  const int slot = WARP ? blockIdx.x * rpb + (threadIdx.x >> 5) : blockIdx.x;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const long step = static_cast<long>(gridDim.x) * rpb;
  const bool full = a.gate == MOE_GATE_FULL, post = (a.flags & MOE_NORM_POST) != 0;
  float acc0[NCH][VEC], acc1[NCH][VEC];
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc0[i][k] = acc1[i][k] = 0.f;
  int turn = 0;
  Chunk<T, VEC> next[5][NCH];
  RowIn next_in = {};
  auto fetch = [&](long row) {
    load_row<T, VEC, NCH>(next[0], a.dz, row, a.ld_z, a.d, tid, tpr);
    load_row<T, VEC, NCH>(next[1], a.dh, row, a.ld_h, a.d, tid, tpr);
    load_row<T, VEC, NCH>(next[2], a.zin, row, a.ld_z, a.d, tid, tpr);
    load_row<T, VEC, NCH>(next[3], a.f, row, a.ld_f, a.d, tid, tpr);
    if (full) load_row<T, VEC, NCH>(next[4], a.g, row, a.ld_g, a.d, tid, tpr);
    next_in = row_in<T>(a, row);
  };
  if (slot < a.rows) fetch(slot);
  for (long row = slot; row < a.rows; row += step) {
    Chunk<T, VEC> q[5][NCH];
#pragma unroll
    for (int k = 0; k < 5; ++k)
#pragma unroll
      for (int i = 0; i < NCH; ++i) q[k][i] = next[k][i];
    const RowIn in = next_in;
    if (row + step < a.rows) fetch(row + step);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    // w_post times a channel gate, and a full gate's values
    auto gates = [&](int i, int c, float *w, float *g) {
      weight_chunk<T, VEC>(a.w_post, c, w);
      weight_chunk<T, VEC>(a.gate == MOE_GATE_CHANNEL ? a.g : nullptr, c, g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        w[k] *= g[k];
        g[k] = 1.f;
      }
      if (full) q[4][i].get(g);
    };
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (tid + i * tpr) * VEC;
      if (c < a.d) {
        float dz[VEC], dh[VEC], z[VEC], f[VEC], w[VEC], wp[VEC], g[VEC];
        q[0][i].get(dz);
        q[1][i].get(dh);
        q[2][i].get(z);
        q[3][i].get(f);
        weight_chunk<T, VEC>(a.w_pre, c, wp);
        gates(i, c, w, g);
#pragma unroll
        for (int k = 0; k < VEC; ++k) add_sums(dz[k], dh[k] * wp[k], z[k], w[k] * g[k] * f[k], s);
      }
    }
    row_sum<WARP, 4>(s, red, turn);
    const RowTerms t = row_terms<T>(a, post, row, in, s, inv_d, tid == 0);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (tid + i * tpr) * VEC;
      if (c < a.d) {
        float dz[VEC], dh[VEC], z[VEC], f[VEC], w[VEC], wp[VEC], g[VEC];
        q[0][i].get(dz);
        q[1][i].get(dh);
        q[2][i].get(z);
        q[3][i].get(f);
        weight_chunk<T, VEC>(a.w_pre, c, wp);
        gates(i, c, w, g);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const ElemOut o =
              elem_out(t, post, a.alpha, dz[k], dh[k], z[k], f[k], wp[k], w[k], g[k], acc0[i][k], acc1[i][k]);
          dz[k] = o.dx;
          dh[k] = o.df;
          z[k] = o.dg;
        }
        if (a.dx) Chunk<T, VEC>::store(static_cast<T *>(a.dx) + row * a.ld_x + c, dz);
        if (a.df) Chunk<T, VEC>::store(static_cast<T *>(a.df) + row * a.ld_f + c, dh);
        if (full && a.dg) Chunk<T, VEC>::store(static_cast<T *>(a.dg) + row * a.ld_g + c, z);
      }
    }
  }
  if (!a.part) return;
  const long ld_p = norm_part_row(a.d);
  float *p = a.part + blockIdx.x * 2 * ld_p;
  if constexpr (WARP) {
    // the block's warps join their column sums in order
    __shared__ float join[2][32 * VEC * NCH];
    for (int turn_of = 0; turn_of < rpb; ++turn_of) {
      if (turn_of == static_cast<int>(threadIdx.x >> 5)) {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
          for (int k = 0; k < VEC; ++k) {
            const int c = (tid + i * tpr) * VEC + k;
            join[0][c] = turn_of ? join[0][c] + acc0[i][k] : acc0[i][k];
            join[1][c] = turn_of ? join[1][c] + acc1[i][k] : acc1[i][k];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
      p[c] = join[0][c];
      p[ld_p + c] = join[1][c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (tid + i * tpr) * VEC;
      if (c < a.d) {
        put_sums<VEC>(p + c, acc0[i]);
        put_sums<VEC>(p + ld_p + c, acc1[i]);
      }
    }
  }
}

// Long rows in two launches that each read the row: the first leaves every row's
// terms in the workspace, the second has no sums over rows left to wait for, so a
// thread keeps its columns for many rows.  10 instead of 6 elements move per
// column, but a row need not fit a block.
template <typename T, int VEC>
__global__ void __launch_bounds__(512) norm_bwd_rows_kernel(const NormArgs a) {
  __shared__ float red[2][4][kMaxWarps];
  const float inv_d = 1.f / static_cast<float>(a.d);
  const bool post = (a.flags & MOE_NORM_POST) != 0;
  int turn = 0;
  for (long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const RowIn in = row_in<T>(a, row);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = threadIdx.x * VEC; c < a.d; c += blockDim.x * VEC) {
      float v[4][VEC], w[VEC], wp[VEC], g[VEC];
      const void *base[4] = {a.dz, a.dh, a.zin, a.f};
      const long ld[4] = {a.ld_z, a.ld_h, a.ld_z, a.ld_f};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        Chunk<T, VEC> q;
        q.clear();
        if (base[t]) q.load(static_cast<const T *>(base[t]) + row * ld[t] + c);
        q.get(v[t]);
      }
      weight_chunk<T, VEC>(a.w_pre, c, wp);
      weight_chunk<T, VEC>(a.w_post, c, w);
      gate_chunk<T, VEC>(a, row, c, 1.f, g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) add_sums(v[0][k], v[1][k] * wp[k], v[2][k], w[k] * g[k] * v[3][k], s);
    }
    row_sum<false, 4>(s, red, turn);
    const RowTerms t = row_terms<T>(a, post, row, in, s, inv_d, threadIdx.x == 0);
    if (threadIdx.x == 0) reinterpret_cast<float4 *>(a.terms)[row] = make_float4(t.rp, t.c1, t.a1, t.c2);
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(128) norm_bwd_apply_kernel(const NormArgs a, int rows_each) {
  pdl_trigger();
  const int c = (blockIdx.x * 128 + threadIdx.x) * VEC;
  if (c >= a.d) return;
  const bool full = a.gate == MOE_GATE_FULL, post = (a.flags & MOE_NORM_POST) != 0;
  float w[VEC], wp[VEC], acc0[VEC], acc1[VEC];
  weight_chunk<T, VEC>(a.w_pre, c, wp);
  weight_chunk<T, VEC>(a.w_post, c, w);
  if (a.gate == MOE_GATE_CHANNEL) {
    float g[VEC];
    weight_chunk<T, VEC>(a.g, c, g);
#pragma unroll
    for (int k = 0; k < VEC; ++k) w[k] *= g[k];
  }
#pragma unroll
  for (int k = 0; k < VEC; ++k) acc0[k] = acc1[k] = 0.f;
  const long first = static_cast<long>(blockIdx.y) * rows_each;
  const long end = first + rows_each < a.rows ? first + rows_each : a.rows;
  constexpr int U = 2;  // rows in flight
  for (long r0 = first; r0 < end; r0 += U) {
    Chunk<T, VEC> q[U][5];
    float4 term[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int t = 0; t < 5; ++t) q[u][t].clear();
      const long row = r0 + u;
      if (row >= end) continue;
      term[u] = reinterpret_cast<const float4 *>(a.terms)[row];
      if (a.dz) q[u][0].load(static_cast<const T *>(a.dz) + row * a.ld_z + c);
      if (a.dh) q[u][1].load(static_cast<const T *>(a.dh) + row * a.ld_h + c);
      if (a.zin) q[u][2].load(static_cast<const T *>(a.zin) + row * a.ld_z + c);
      if (a.f) q[u][3].load(static_cast<const T *>(a.f) + row * a.ld_f + c);
      if (full) q[u][4].load(static_cast<const T *>(a.g) + row * a.ld_g + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long row = r0 + u;
      if (row >= end) break;
      const RowTerms t = {term[u].x, term[u].y, term[u].z, term[u].w};
      float dz[VEC], dh[VEC], z[VEC], f[VEC], g[VEC];
      q[u][0].get(dz);
      q[u][1].get(dh);
      q[u][2].get(z);
      q[u][3].get(f);
      q[u][4].get(g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const ElemOut o =
            elem_out(t, post, a.alpha, dz[k], dh[k], z[k], f[k], wp[k], w[k], full ? g[k] : 1.f, acc0[k], acc1[k]);
        dz[k] = o.dx;
        f[k] = o.df;
        z[k] = o.dg;
      }
      if (a.dx) Chunk<T, VEC>::store(static_cast<T *>(a.dx) + row * a.ld_x + c, dz);
      if (a.df) Chunk<T, VEC>::store(static_cast<T *>(a.df) + row * a.ld_f + c, f);
      if (full && a.dg) Chunk<T, VEC>::store(static_cast<T *>(a.dg) + row * a.ld_g + c, z);
    }
  }
  if (a.part) {
    const long ld_p = norm_part_row(a.d);
    float *p = a.part + blockIdx.y * 2 * ld_p + c;
    put_sums<VEC>(p, acc0);
    put_sums<VEC>(p + ld_p, acc1);
  }
}

template <typename T, int VEC>
cudaError_t bwd_long(const NormArgs &a, int num_sms, int *slots, cudaStream_t s) {
  norm_bwd_rows_kernel<T, VEC><<<a.rows < num_sms * 4L ? a.rows : num_sms * 4, 512, 0, s>>>(a);
  const int tiles = (a.d + 128 * VEC - 1) / (128 * VEC);
  long groups = (num_sms * 16L + tiles - 1) / tiles;
  if (groups > norm_max_blocks(a.d)) groups = norm_max_blocks(a.d);
  if (groups > a.rows) groups = a.rows;
  const int each = static_cast<int>((a.rows + groups - 1) / groups);
  groups = (a.rows + each - 1) / each;
  *slots = static_cast<int>(groups);
  norm_bwd_apply_kernel<T, VEC><<<dim3(tiles, static_cast<unsigned>(groups)), 128, 0, s>>>(a, each);
  return cudaGetLastError();
}

// dw_pre, dw_post and a channel gate's gradient from the blocks' column sums:
// 32 columns per block, the partial rows in 32 interleaved runs joined in order.
// Where the rows start inside a 16-byte chunk (`mod` elements further into one with
// every row), so do the partial rows, block b's like row b.
template <typename T>
__global__ void __launch_bounds__(1024) norm_columns_kernel(const NormArgs a, int slots, int mod) {
  __shared__ float sh[32][32];
  const long ld_p = norm_part_row(a.d);
  pdl_wait();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5, k = blockIdx.y;
  float v = 0.f;
  if (c < a.d)
    for (int b = run; b < slots; b += 32) v += a.part[(b * 2L + k) * ld_p + c + row_shift<T>(mod, b)];
  sh[run][threadIdx.x & 31] = v;
  __syncthreads();
  if (run || c >= a.d) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) v += sh[i][threadIdx.x];
  if (k == 0) {
    if (a.dw_pre) static_cast<T *>(a.dw_pre)[c] = Elem<T>::from(v);
    return;
  }
  float w = 1.f, g = 1.f;
  if (a.w_post) w = Elem<T>::to(static_cast<const T *>(a.w_post)[c]);
  if (a.gate == MOE_GATE_CHANNEL) g = Elem<T>::to(static_cast<const T *>(a.g)[c]);
  if (a.dw_post) static_cast<T *>(a.dw_post)[c] = Elem<T>::from(g * v);
  if (a.gate == MOE_GATE_CHANNEL && a.dg) static_cast<T *>(a.dg)[c] = Elem<T>::from(w * v);
}

bool vec16(const void *p, long ld, int esz) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * esz) % 16 == 0;
}

int round32(int n) { return (n + 31) / 32 * 32; }

// Rows of 16-byte chunks only when every tensor of the call has them.
template <typename T>
bool all_vec(const NormArgs &a) {
  const int e = sizeof(T);
  return (a.d * e) % 16 == 0 && vec16(a.x, a.ld_x, e) && vec16(a.dx, a.ld_x, e) && vec16(a.f, a.ld_f, e) &&
         vec16(a.df, a.ld_f, e) && vec16(a.z, a.ld_z, e) && vec16(a.zin, a.ld_z, e) && vec16(a.dz, a.ld_z, e) &&
         vec16(a.h, a.ld_h, e) && vec16(a.dh, a.ld_h, e) && vec16(a.w_pre, 0, e) && vec16(a.w_post, 0, e) &&
         (a.gate == MOE_GATE_NONE || a.gate == MOE_GATE_ROW ||
          (vec16(a.g, a.gate == MOE_GATE_FULL ? a.ld_g : 0, e) &&
           (a.gate == MOE_GATE_CHANNEL || vec16(a.dg, a.ld_g, e))));
}

// Blocks of `threads` of a kernel that fit an SM, asked once per device and size.
template <typename K>
int resident(K kernel, int threads, int (&memo)[33][64]) {
  return per_device_memo(memo[threads >> 5], [&]() {
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) == cudaSuccess && n > 0 ? n : 1;
  });
}

template <typename T, int VEC, int NCH, bool WARP, int THREADS, int MINB>
cudaError_t fwd_one(const NormArgs &a, int threads, int num_sms, cudaStream_t s) {
  static int memo[33][64] = {};
  const auto kernel = norm_fwd_kernel<T, VEC, NCH, WARP, THREADS, MINB>;
  const int rpb = WARP ? threads / 32 : 1;
  const long blocks = (a.rows + rpb - 1) / rpb, most = static_cast<long>(num_sms) * resident(kernel, threads, memo);
  kernel<<<static_cast<int>(blocks < most ? blocks : most), threads, 0, s>>>(a);
  return cudaGetLastError();
}

// Columns per thread: 16 of a 16-byte chunked row, 8 of one that is not (each
// takes a register of its own).  Up to 512 columns a warp holds a row, beyond
// a block.
template <typename T, int VEC>
cudaError_t fwd_vec(const NormArgs &a, int num_sms, cudaStream_t s) {
  constexpr int EPT = VEC > 1 ? 16 : 8, NCH = EPT / VEC;
  if (a.d <= 32 * EPT) return fwd_one<T, VEC, NCH, true, 256, 2>(a, 256, num_sms, s);
  const int threads = round32((a.d + EPT - 1) / EPT);
  if (threads <= 256) return fwd_one<T, VEC, NCH, false, 256, 3>(a, threads, num_sms, s);
  if (threads <= 512) return fwd_one<T, VEC, NCH, false, 512, 2>(a, threads, num_sms, s);
  return fwd_one<T, VEC, NCH, false, 1024, 1>(a, threads, num_sms, s);
}

template <typename T>
cudaError_t fwd_type(const NormArgs &a, int num_sms, cudaStream_t s) {
  const bool vec = all_vec<T>(a);
  if (a.rows > num_sms && norm_ring_fits(a, false)) return launch_norm_fwd_ring(a, num_sms, s);
  if (a.d > (vec ? 16384 : 8192)) {
    const int grid = a.rows < 2 * num_sms ? a.rows : 2 * num_sms;
    norm_fwd_long_kernel<T><<<grid, 1024, 0, s>>>(a);
    return cudaGetLastError();
  }
  return vec ? fwd_vec<T, Elem<T>::VEC>(a, num_sms, s) : fwd_vec<T, 1>(a, num_sms, s);
}

template <typename T, int VEC, int NCH, bool WARP, int THREADS, int MINB>
cudaError_t bwd_one(const NormArgs &a, int threads, int num_sms, int *slots, cudaStream_t s) {
  static int memo[33][64] = {};
  const auto kernel = norm_bwd_kernel<T, VEC, NCH, WARP, THREADS, MINB>;
  const int rpb = WARP ? threads / 32 : 1;
  const long blocks = (a.rows + rpb - 1) / rpb;
  long grid = static_cast<long>(num_sms) * resident(kernel, threads, memo);
  if (grid > norm_max_blocks(a.d)) grid = norm_max_blocks(a.d);
  if (blocks < grid) grid = blocks;
  *slots = static_cast<int>(grid);
  kernel<<<static_cast<int>(grid), threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t bwd_vec(const NormArgs &a, int num_sms, int *slots, cudaStream_t s) {
  if constexpr (VEC > 1) {
    constexpr int NCH = 16 / VEC;
    if (a.d <= 256) return bwd_one<T, VEC, NCH / 2, true, 256, 2>(a, 256, num_sms, slots, s);
    if (sizeof(T) == 4 && a.d <= 4096) {  // fp32 rows take twice the registers
      const int threads = round32((a.d + 7) / 8);
      if (threads <= 256) return bwd_one<T, VEC, NCH / 2, false, 256, 2>(a, threads, num_sms, slots, s);
      return bwd_one<T, VEC, NCH / 2, false, 512, 1>(a, threads, num_sms, slots, s);
    }
    const int threads = round32((a.d + 15) / 16);
    if (threads <= 192) return bwd_one<T, VEC, NCH, false, 192, 2>(a, threads, num_sms, slots, s);
    if (threads <= 384) return bwd_one<T, VEC, NCH, false, 384, 1>(a, threads, num_sms, slots, s);
    return bwd_one<T, VEC, NCH, false, 512, 1>(a, threads, num_sms, slots, s);
  } else {
    if (a.d <= 128) return bwd_one<T, 1, 4, true, 256, 2>(a, 256, num_sms, slots, s);
    const int threads = round32((a.d + 3) / 4);
    if (threads <= 256) return bwd_one<T, 1, 4, false, 256, 4>(a, threads, num_sms, slots, s);
    if (threads <= 512) return bwd_one<T, 1, 4, false, 512, 2>(a, threads, num_sms, slots, s);
    if (threads <= 1024) return bwd_one<T, 1, 4, false, 1024, 1>(a, threads, num_sms, slots, s);
    return bwd_one<T, 1, 8, false, 1024, 1>(a, round32((a.d + 7) / 8), num_sms, slots, s);
  }
}

template <typename T>
cudaError_t bwd_type(const NormArgs &a, int num_sms, cudaStream_t s) {
  int slots = 0, mod = 0;
  if (a.rows > 0) {
    cudaError_t e;
    HostTrace t("norm_backward", s);
    const bool vec = all_vec<T>(a);
    if (a.rows > num_sms && norm_ring_fits(a, true)) {
      e = launch_norm_bwd_ring(a, num_sms, &slots, s);
      mod = static_cast<int>(a.ld_z % Elem<T>::VEC);
    } else if (a.d > norm_long(a.dtype)) {
      e = vec ? bwd_long<T, Elem<T>::VEC>(a, num_sms, &slots, s) : bwd_long<T, 1>(a, num_sms, &slots, s);
    } else {
      e = vec ? bwd_vec<T, Elem<T>::VEC>(a, num_sms, &slots, s) : bwd_vec<T, 1>(a, num_sms, &slots, s);
    }
    if (e != cudaSuccess) return e;
  }
  if (!a.part) return cudaSuccess;
  HostTrace t("norm_columns", s);
  const dim3 grid((a.d + 31) / 32, 2);
  if (a.rows > 0) return launch_early(norm_columns_kernel<T>, grid, 1024, s, a, slots, mod);
  norm_columns_kernel<T><<<grid, 1024, 0, s>>>(a, slots, mod);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs &a, int num_sms, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  HostTrace t("norm_forward", s);
  switch (a.dtype) {
    case MOE_ELEM_BF16: return fwd_type<__nv_bfloat16>(a, num_sms, s);
    case MOE_ELEM_FP16: return fwd_type<__half>(a, num_sms, s);
    default: return fwd_type<float>(a, num_sms, s);
  }
}

cudaError_t launch_norm_backward(const NormArgs &a, int num_sms, cudaStream_t s) {
  switch (a.dtype) {
    case MOE_ELEM_BF16: return bwd_type<__nv_bfloat16>(a, num_sms, s);
    case MOE_ELEM_FP16: return bwd_type<__half>(a, num_sms, s);
    default: return bwd_type<float>(a, num_sms, s);
  }
}

}  // namespace moe
