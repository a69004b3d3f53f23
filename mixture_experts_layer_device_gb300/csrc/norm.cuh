// Pieces shared by the norm kernels: the sum over a row's threads, chunked
// access to rows, and the backward's per-row terms.
#pragma once

#include "block.h"
#include "elem.cuh"

namespace moe {

namespace {

constexpr int kMaxWarps = 32;

// Sums of N values over a warp: lanes first trade values for lanes (each halving
// of the values costs one shuffle per value kept), so N sums cost N - 1 +
// 5 - log2 N shuffles instead of 5 N.  Returns the sum of value
// (lane / (32 / N)); fixed order.
template <int N>
MOE_DEV float warp_sums(const float *in, int lane) {
  float v[N];
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = in[k];
  int o = 16;
#pragma unroll
  for (int n = N; n > 1; n >>= 1, o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int k = 0; k < n / 2; ++k) {
      const float give = up ? v[k] : v[k + n / 2], keep = up ? v[k + n / 2] : v[k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// The same over a block in two steps, with a barrier of the caller's between them:
// each warp's sums into red[N][32], then every thread takes the totals.
template <int N>
MOE_DEV void block_sums_put(const float *v, float (*red)[kMaxWarps]) {
  constexpr int SHARE = 32 / N;
  const int lane = threadIdx.x & 31;
  const float t = warp_sums<N>(v, lane);
  if (lane % SHARE == 0) red[lane / SHARE][threadIdx.x >> 5] = t;
}
template <int N>
MOE_DEV void block_sums_get(float *v, const float (*red)[kMaxWarps]) {
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = lane < nw ? red[k][lane] : 0.f;
  const float t = warp_sums<N>(v, lane);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = N > 1 ? __shfl_sync(0xffffffffu, t, k * (32 / N)) : t;
}

// Sums over the threads that share a row, left in every one of them: a warp
// (WARP), or the block through red[2][N][32] (two buffers in turn: one barrier
// per call).  Fixed order.
template <bool WARP, int N>
MOE_DEV void row_sum(float *v, float (*red)[N][kMaxWarps], int &turn) {
  if constexpr (WARP) {
    const float t = warp_sums<N>(v, threadIdx.x & 31);
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = N > 1 ? __shfl_sync(0xffffffffu, t, k * (32 / N)) : t;
  } else {
    block_sums_put<N>(v, red[turn]);
    __syncthreads();
    block_sums_get<N>(v, red[turn]);
    turn ^= 1;
  }
}

// VEC elements of a row at p (16 bytes at once when VEC > 1).
template <typename T, int VEC>
struct Chunk {
  uint4 q;
  MOE_DEV void load(const T *p) { q = ld_stream(p); }
  MOE_DEV void load_cached(const T *p) { q = __ldg(reinterpret_cast<const uint4 *>(p)); }
  MOE_DEV void clear() { q = make_uint4(0, 0, 0, 0); }
  MOE_DEV void get(float *v) const { Elem<T>::unpack(q, v); }
  MOE_DEV static void store(T *p, const float *v) { st_stream(p, Elem<T>::pack(v)); }
};
template <typename T>
struct Chunk<T, 1> {
  T q;
  MOE_DEV void load(const T *p) { q = *p; }
  MOE_DEV void load_cached(const T *p) { q = *p; }
  MOE_DEV void clear() { q = Elem<T>::from(0.f); }
  MOE_DEV void get(float *v) const { v[0] = Elem<T>::to(q); }
  MOE_DEV static void store(T *p, const float *v) { *p = Elem<T>::from(v[0]); }
};

template <typename T, int VEC>
MOE_DEV void weight_chunk(const void *w, long at, float *v) {
  if (w) {
    Chunk<T, VEC> q;
    q.load_cached(static_cast<const T *>(w) + at);
    q.get(v);
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = 1.f;
  }
}

// The gate of VEC columns of a row (ROW's value comes in as `row_gate`).
template <typename T, int VEC>
MOE_DEV void gate_chunk(const NormArgs &a, long row, int c, float row_gate, float *v) {
  if (a.gate == MOE_GATE_CHANNEL) {
    weight_chunk<T, VEC>(a.g, c, v);
  } else if (a.gate == MOE_GATE_FULL) {
    Chunk<T, VEC> q;
    q.load(static_cast<const T *>(a.g) + row * a.ld_g + c);
    q.get(v);
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = row_gate;
  }
}

template <typename T>
MOE_DEV float row_gate_of(const NormArgs &a, long row) {
  return a.gate == MOE_GATE_ROW ? Elem<T>::to(static_cast<const T *>(a.g)[row]) : 1.f;
}

// ---------------------------------------------------------------- backward terms
// Per-row inputs of the backward: r_pre (0 without the pre norm), r_post (1
// without the post norm) and the row gate (1 without one).
struct RowIn {
  float rp, rq, rg;
};
template <typename T>
MOE_DEV RowIn row_in(const NormArgs &a, long row) {
  RowIn t;
  t.rp = (a.flags & MOE_NORM_PRE) ? __ldg(a.r_pre_in + row) : 0.f;
  t.rq = (a.flags & MOE_NORM_POST) ? __ldg(a.r_post_in + row) : 1.f;
  t.rg = row_gate_of<T>(a, row);
  return t;
}

// What a row's columns need once its sums are known, from
//   s[0] <w_pre dh, z>, s[1] <dz, q>, s[2] <w_pre dh, q>, s[3] <z, q>
// with q = w_post g f, g without a row gate:
//   t = dz + rp (w_pre dh) - c1 (rp z),   c1 = rp^2 s[0] / d
//   df = a1 (w_post g t) - c2 (a1 f),     a1 = rq rg, c2 = rq^2 <t, q> / d
// Multiplied in this order no factor leaves fp32 before the roots' own squares do
// (rq^3 would at |f| of 1e13).  Also writes a row gate's gradient <t, n>.
struct RowTerms {
  float rp, c1, a1, c2;
};
template <typename T>
MOE_DEV RowTerms row_terms(const NormArgs &a, bool post, long row, const RowIn &in, const float *s, float inv_d,
                           bool first) {
  RowTerms t;
  t.rp = in.rp;
  t.c1 = in.rp * (in.rp * (s[0] * inv_d));
  float tq = s[1] + in.rp * (s[2] - t.c1 * s[3]);  // <t, q>
  if (!post && !(a.flags & MOE_NORM_PRE)) tq = s[1];  // f may be infinite: no 0 * inf of the terms that are not there
  t.a1 = in.rq * in.rg;
  t.c2 = post ? in.rq * (in.rq * (tq * inv_d)) : 0.f;
  if (a.gate == MOE_GATE_ROW && a.dg && first) static_cast<T *>(a.dg)[row] = Elem<T>::from(tq * in.rq);
  return t;
}

// One element's share of the row sums; dhw = w_pre dh.
MOE_DEV void add_sums(float dz, float dhw, float z, float q, float *s) {
  s[0] = fmaf(dhw, z, s[0]);
  s[1] = fmaf(dz, q, s[1]);
  s[2] = fmaf(dhw, q, s[2]);
  s[3] = fmaf(z, q, s[3]);
}

// One element after the sums.  w = w_post times a channel gate; g = a full
// gate's value, else 1.  acc0 sums dh z r_pre (dw_pre); acc1 sums t f r_post
// with a row or full gate (dw_post, and a channel gate's gradient).  Without the
// post norm df does not depend on f, which may be infinite then.
struct ElemOut {
  float dx, df, dg;
};
MOE_DEV ElemOut elem_out(const RowTerms &t, bool post, float alpha, float dz, float dh, float z, float f, float wp,
                         float w, float g, float &acc0, float &acc1) {
  ElemOut o;
  const float y = t.rp * z;
  const float tt = fmaf(t.rp, dh * wp, fmaf(-t.c1, y, dz));
  acc0 = fmaf(dh, y, acc0);
  const float nh = f * t.a1, tg = tt * g, tw = tt * w;
  acc1 = fmaf(tg, nh, acc1);
  o.dx = alpha * tt;
  o.dg = tw * nh;
  o.df = fmaf(t.a1, tw * g, post ? -(t.c2 * nh) : 0.f);
  return o;
}

}  // namespace

// Kernels with rows in flight through shared memory (norm_ring.cu), for more rows
// than SMs; false when they do not take the call's rows.
bool norm_ring_fits(const NormArgs &a, bool backward);
cudaError_t launch_norm_fwd_ring(const NormArgs &a, int num_sms, cudaStream_t s);
cudaError_t launch_norm_bwd_ring(const NormArgs &a, int num_sms, int *slots, cudaStream_t s);

// How far into a 16-byte chunk the rows of block b start, in elements.
template <typename T>
MOE_DEV int row_shift(long ld, long row) {
  return static_cast<int>((row % Elem<T>::VEC) * (ld % Elem<T>::VEC) % Elem<T>::VEC);
}

// One thread's column sums into a partial row.
template <int VEC>
MOE_DEV void put_sums(float *p, const float *v) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int k = 0; k < VEC; k += 4) *reinterpret_cast<float4 *>(p + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) p[k] = v[k];
  }
}

}  // namespace moe
