// The loss over a vocabulary, without its logits in memory: the rows that count,
// the copy of x that the products read, and what joins the products' parts.
//   z_tv = x_t . w_v,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t[label_t]
//   dz_tv = (dloss_t + dlse_t) exp(z_tv - lse_t) - dloss_t [v = label_t]
//   dx_t = sum_v dz_tv w_v,  dw_v = sum_t dz_tv x_t
// The products are in vocab_tc.cu.
#include "block.h"
#include "elem.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

MOE_DEV long label_of(const VocabArgs &a, int t) {
  return a.labels64 ? static_cast<long>(static_cast<const long long *>(a.labels)[t])
                    : static_cast<long>(static_cast<const int *>(a.labels)[t]);
}

// ---------------------------------------------------------------- rows that count
// One block: the rows that count, in order.  Forward: those whose label lies in the
// vocabulary; the others' loss and lse are zero.  Backward: of those, the ones that
// have a gradient at all.  What is rounded to 16 bits, dz, is held relative to the
// largest coefficient of all rows (times 2^14 in fp16, whose smallest steps
// probabilities would sink below): equal coefficients, as a mean gives, are then 1
// and lose nothing; *scale undoes it.
constexpr int kRowThreads = 1024, kRowItems = 8;

// The labels (-1: a row that does not count) and coefficients of kRowItems rows, 32 apart
// from `first` on (a warp has 32 kRowItems rows next to each other), all loads in flight
// together; the rows that count as a mask.
template <bool BACKWARD>
struct RowItems {
  int label[kRowItems];
  float p[kRowItems], l[kRowItems];
  MOE_DEV unsigned load(const VocabArgs &a, int first) {
    long lab[kRowItems];
#pragma unroll
    for (int k = 0; k < kRowItems; ++k) {
      const int t = first + 32 * k;
      const bool has = t < a.rows;
      lab[k] = has ? label_of(a, t) : -1;
      l[k] = BACKWARD && has && a.dloss ? a.dloss[t] : 0.f;
      p[k] = BACKWARD && has && a.dlse ? a.dlse[t] : 0.f;
    }
    unsigned mask = 0;
#pragma unroll
    for (int k = 0; k < kRowItems; ++k) {
      p[k] += l[k];
      const bool counts = lab[k] >= 0 && lab[k] < a.V && (!BACKWARD || p[k] != 0.f || l[k] != 0.f);  // NaN counts
      label[k] = counts ? static_cast<int>(lab[k]) : -1;
      mask |= counts ? 1u << k : 0u;
    }
    return mask;
  }
  // the largest coefficient; one that is not finite keeps to its own row
  MOE_DEV float top(unsigned mask) const {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kRowItems; ++k) {
      const float m = fmaxf(fabsf(p[k]), fabsf(l[k]));
      if ((mask >> k & 1u) && m <= 3.402823466e38f) t = fmaxf(t, m);
    }
    return t;
  }
  // row t, item k, counts and stands at place `at`
  MOE_DEV void write(const VocabArgs &a, int k, int t, int at, float top, float up) const {
    a.row[at] = t;
    a.label[at] = label[k];
    if constexpr (BACKWARD) {
      a.place[t] = at;
      a.coef_p[at] = p[k] / top * up;
      a.coef_l[at] = l[k] / top * up;
      a.base[at] = a.lse_in[t] * kLog2e;
    }
  }
  MOE_DEV void leave_out(const VocabArgs &a, int t) const {
    if constexpr (BACKWARD) {
      a.place[t] = -1;
    } else {
      a.loss[t] = 0.f;
      a.lse[t] = 0.f;
    }
  }
};

MOE_DEV float scale_up(const VocabArgs &a) { return a.dtype == MOE_ELEM_FP16 ? 16384.f : 1.f; }

template <bool BACKWARD>
MOE_DEV void finish_rows(const VocabArgs &a, int n, float top, float up) {
  *a.status = 0;
  *a.count = n;
  if constexpr (BACKWARD) *a.scale = top / up;
}

// Places behind the last one: no label, no gradient.
template <bool BACKWARD, int THREADS>
MOE_DEV void pad_rows(const VocabArgs &a, int n) {
  for (int i = n + threadIdx.x; i < ((n + 255) & ~255); i += THREADS) {
    a.label[i] = -1;
    if constexpr (BACKWARD) a.coef_p[i] = a.coef_l[i] = a.base[i] = 0.f;
  }
}

template <bool BACKWARD>
__global__ void __launch_bounds__(kRowThreads) vocab_rows_kernel(const VocabArgs a) {
  pdl_trigger();
  __shared__ int warps[32];
  __shared__ float tops[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  RowItems<BACKWARD> r;
  float top = 0.f;
  if constexpr (BACKWARD) {
    for (int t0 = 0; t0 < a.rows; t0 += kRowThreads * kRowItems) {
      const unsigned mask = r.load(a, t0 + warp * 32 * kRowItems + lane);
      top = fmaxf(top, r.top(mask));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = tops[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == 0.f) top = 1.f;
  }
  const float up = scale_up(a);
  int done = 0;
  for (int t0 = 0; t0 < a.rows; t0 += kRowThreads * kRowItems) {
    const int first = t0 + warp * 32 * kRowItems + lane;
    const unsigned mask = r.load(a, first);
    const int mine = __reduce_add_sync(0xffffffffu, __popc(mask));
    __syncthreads();
    if (lane == 0) warps[warp] = mine;
    __syncthreads();
    const int w = warps[lane];
    int base = done + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    done += __reduce_add_sync(0xffffffffu, w);
#pragma unroll
    for (int k = 0; k < kRowItems; ++k) {
      const int t = first + 32 * k;
      const unsigned same = __ballot_sync(0xffffffffu, mask >> k & 1u);
      const int at = base + __popc(same & ((1u << lane) - 1));
      base += __popc(same);
      if (t >= a.rows) continue;
      if (mask >> k & 1u) r.write(a, k, t, at, top, up);
      else r.leave_out(a, t);
    }
  }
  if (threadIdx.x == 0) finish_rows<BACKWARD>(a, done, top, up);
  pad_rows<BACKWARD, kRowThreads>(a, done);
}

// ---------------------------------------------------------------- copies
// xs [count rounded up to 128][ld_xs] = x[row[i]], zeros beyond x's columns and behind
// the last row: a sum over rows takes them in steps of up to 128.  TMA could fill those
// zeros in, but boxes that lie half outside their tensor cost it time: one row and 131072
// entries of 7168 take 508 us with such boxes, 256 rows 338 us.
// On the way the label's logit, a dot product in fp32 whose terms are rounded to
// nearest.  The tensor cores' sums truncate: at d = 7168 their logits are off by some
// 4e-6 of their size, which the loss of a row that is sure of its label would consist of.
// GROUP threads per row: 32, or the block's 256 from 2048 columns on (31 rows of 8192: 9.9
// us, 16.0 with 32; 16384 rows of 512: 9.7 with 32, 20.0 with 256; of 2048: 25 and 28).
constexpr int kWideRow = 2048;

template <typename T>
MOE_DEV uint4 eight(const T *p, int left, bool vec) {
  if (vec) return *reinterpret_cast<const uint4 *>(p);
  const uint16_t *e = reinterpret_cast<const uint16_t *>(p);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t lo = 2 * k < left ? e[2 * k] : 0u, hi = 2 * k + 1 < left ? e[2 * k + 1] : 0u;
    w[k] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a row needs of the rows kernel, in global memory or, where the gather has found the
// rows itself, in shared memory.
struct RowList {
  const int *row, *label;
  const float *p, *l;
  int n;
};

template <typename T, int GROUP, bool BACKWARD>
MOE_DEV void gather_rows(const VocabArgs &a, const RowList &list) {
  __shared__ float part[8];
  const int n = list.n, chunks = static_cast<int>(a.ld_xs >> 3);
  const int end = (n + 127) & ~127;
  const bool vec_x = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && a.ld_x % 8 == 0 && a.d % 8 == 0;
  const bool vec_w = (reinterpret_cast<uintptr_t>(a.w) & 15) == 0 && a.ld_w % 8 == 0 && a.d % 8 == 0;
  const int me = threadIdx.x % GROUP, warp = threadIdx.x >> 5;
  for (long i = static_cast<long>(blockIdx.x) * (256 / GROUP) + threadIdx.x / GROUP; i < end;
       i += static_cast<long>(gridDim.x) * (256 / GROUP)) {
    uint4 *to = reinterpret_cast<uint4 *>(static_cast<T *>(a.xs) + i * a.ld_xs);
    if (i >= n) {
      for (int c = me; c < chunks; c += GROUP) to[c] = make_uint4(0, 0, 0, 0);
      continue;  // of whole groups; with GROUP 256 of the whole block
    }
    const int label = list.label[i], from = list.row[i];
    const T *x = static_cast<const T *>(a.x) + from * a.ld_x;
    const T *w = static_cast<const T *>(a.w) + label * a.ld_w;
    float s = 0.f;
#pragma unroll 2
    for (int c = me; c < chunks; c += GROUP) {
      const uint4 q = eight(x + c * 8, a.d - c * 8, vec_x), r = eight(w + c * 8, a.d - c * 8, vec_w);
      to[c] = q;
      float u[8], v[8];
      Elem<T>::unpack(q, u);
      Elem<T>::unpack(r, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(u[k], v[k], s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if constexpr (GROUP == 256) {
      __syncthreads();
      if ((threadIdx.x & 31) == 0) part[warp] = s;
      __syncthreads();
      s = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += part[k];
    }
    if (me == 0) {
      if constexpr (BACKWARD) {
        // the label's dz: coef_p exp(z - lse) - coef_l, without losing it where exp is near 1
        const float p = list.p[i], l = list.l[i];
        a.hit[i] = p == 0.f ? -l : (p - l) + p * expm1f(s - a.lse_in[from]);
      } else {
        a.hit[i] = s;
      }
    }
  }
}

template <typename T, int GROUP, bool BACKWARD>
__global__ void __launch_bounds__(256) vocab_gather_kernel(const VocabArgs a) {
  pdl_wait();
  pdl_trigger();
  gather_rows<T, GROUP, BACKWARD>(a, RowList{a.row, a.label, a.coef_p, a.coef_l, *a.count});
}

// Up to 256 kRowItems rows: every block finds the rows that count itself (block 0 writes
// them down), which saves a launch (31 rows, 1000 entries of 256: 24.4 us a
// call, 26.4 in two).
template <typename T, int GROUP, bool BACKWARD>
__global__ void __launch_bounds__(256) vocab_rows_gather_kernel(const VocabArgs a) {
  constexpr int MOST = 256 * kRowItems;
  __shared__ int row[MOST], label[MOST], warps[8];
  __shared__ float p[BACKWARD ? MOST : 1], l[BACKWARD ? MOST : 1], tops[8];
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool writes = blockIdx.x == 0;
  RowItems<BACKWARD> r;
  const int first = warp * 32 * kRowItems + lane;
  const unsigned mask = r.load(a, first);
  float top = 0.f;
  if constexpr (BACKWARD) top = r.top(mask);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int mine = __reduce_add_sync(0xffffffffu, __popc(mask));
  if (lane == 0) {
    warps[warp] = mine;
    tops[warp] = top;
  }
  __syncthreads();
  int base = 0, n = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) base += warps[w];
    n += warps[w];
    top = fmaxf(top, tops[w]);
  }
  if (top == 0.f) top = 1.f;
  const float up = scale_up(a);
#pragma unroll
  for (int k = 0; k < kRowItems; ++k) {
    const int t = first + 32 * k;
    const unsigned same = __ballot_sync(0xffffffffu, mask >> k & 1u);
    const int at = base + __popc(same & ((1u << lane) - 1));
    base += __popc(same);
    if (t >= a.rows) continue;
    if (mask >> k & 1u) {
      row[at] = t;
      label[at] = r.label[k];
      if constexpr (BACKWARD) {
        p[at] = r.p[k] / top * up;
        l[at] = r.l[k] / top * up;
      }
      if (writes) r.write(a, k, t, at, top, up);
    } else if (writes) {
      r.leave_out(a, t);
    }
  }
  if (writes) {
    if (threadIdx.x == 0) finish_rows<BACKWARD>(a, n, top, up);
    pad_rows<BACKWARD, 256>(a, n);
  }
  __syncthreads();
  gather_rows<T, GROUP, BACKWARD>(a, RowList{row, label, p, l, n});
}

// w's rows into rows that TMA can address: a thread per 8 elements (50001 x 321: 20 us; a
// warp per row, lanes on neighbouring words, 28 us; by way of shared memory 20 to 25).
__global__ void __launch_bounds__(256) vocab_pad_kernel(const VocabArgs a) {
  const int chunks = static_cast<int>(a.ld_ws_w >> 3);
  const long total = static_cast<long>(a.V) * chunks;
  for (long u = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; u < total; u += static_cast<long>(gridDim.x) * 256) {
    const long v = u / chunks;
    const int c = static_cast<int>(u - v * chunks) * 8;
    const uint16_t *p = static_cast<const uint16_t *>(a.w) + v * a.ld_w + c;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = c + 2 * k < a.d ? p[2 * k] : 0u, hi = c + 2 * k + 1 < a.d ? p[2 * k + 1] : 0u;
      w[k] = lo | (hi << 16);
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.ws_w) + v * a.ld_ws_w + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---------------------------------------------------------------- joins
// Parts are (maximum, sum of exponentials from it); where a maximum is not finite, from zero.
MOE_DEV float from_of(float m) { return fabsf(m) <= 3.402823466e38f ? m : 0.f; }

// GROUP threads per row that counts: 32, or the block's 256 for few rows with many parts (5
// rows of 1024 parts: 6.0 us, 9.8 with 32; 16384 rows of 8: 8.1 with 32, 26.5 with 256).  The parts hold
// all logits but the label's, z:
//   loss = log(1 + S exp(m - z)),  lse = z + loss
// where that is in range, which keeps a small loss's precision.
template <int GROUP>
__global__ void __launch_bounds__(256) vocab_loss_kernel(const VocabArgs a) {
  __shared__ float tops[8], sums[8];
  pdl_wait();
  const int n = *a.count, me = threadIdx.x % GROUP, warp = threadIdx.x >> 5;
  for (int i = blockIdx.x * (256 / GROUP) + threadIdx.x / GROUP; i < n; i += gridDim.x * (256 / GROUP)) {
    const float2 *p = a.part + static_cast<long>(i) * a.parts;
    float top = -__int_as_float(0x7f800000), s = 0.f;
#pragma unroll 4
    for (int k = me; k < a.parts; k += GROUP) top = fmaxf(top, p[k].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if constexpr (GROUP == 256) {
      if ((threadIdx.x & 31) == 0) tops[warp] = top;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) top = fmaxf(top, tops[k]);
    }
    const float from = from_of(top);
#pragma unroll 4
    for (int k = me; k < a.parts; k += GROUP) {
      const float2 v = p[k];  // a part without logits has sum 0
      s += v.y == 0.f ? 0.f : v.y * exp2f((from_of(v.x) - from) * kLog2e);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if constexpr (GROUP == 256) {
      if ((threadIdx.x & 31) == 0) sums[warp] = s;
      __syncthreads();
      s = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += sums[k];
    }
    if (me == 0) {
      const float z = a.hit[i], others = from + logf(s);  // -inf: the label is alone
      float loss, lse;
      if (others <= z) {
        const bool infinite = fabsf(z) > 3.402823466e38f;  // lse is z, and z - z no number
        loss = infinite ? z - z : log1pf(expf(others - z));
        lse = infinite ? z : z + loss;
      } else {  // also where another logit is not finite, or one is NaN
        lse = others + log1pf(expf(z - others));
        loss = lse - z;
      }
      const int t = a.row[i];
      a.lse[t] = lse;
      a.loss[t] = loss;
    }
    if constexpr (GROUP == 256) __syncthreads();  // the shared values have been read
  }
}

// dx of every row: the splits' sums in order, times *scale; zeros for rows that do not
// count.
template <typename T>
__global__ void __launch_bounds__(256) vocab_dx_kernel(const VocabArgs a, bool vec) {
  pdl_wait();
  const float scale = *a.scale;
  const int chunks = (a.d + 7) >> 3;
  const long total = static_cast<long>(a.rows) * chunks, step = static_cast<long>(a.rows) * a.ld_sum;
  for (long u = static_cast<long>(blockIdx.x) * 256 + threadIdx.x; u < total; u += static_cast<long>(gridDim.x) * 256) {
    const int t = static_cast<int>(u / chunks), c = static_cast<int>(u - static_cast<long>(t) * chunks) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int i = a.place[t];
    if (i >= 0) {
      const float *p = a.sum + i * a.ld_sum + c;
#pragma unroll 4
      for (int k = 0; k < a.splits; ++k, p += step) {
        const float4 lo = *reinterpret_cast<const float4 *>(p), hi = *reinterpret_cast<const float4 *>(p + 4);
        v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
        v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= scale;
    }
    T *o = static_cast<T *>(a.dx) + t * a.ld_dx + c;
    if (vec) {
      *reinterpret_cast<uint4 *>(o) = Elem<T>::pack(v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < a.d) o[k] = Elem<T>::from(v[k]);
    }
  }
}

unsigned blocks_of(long threads, int num_sms) {
  const long want = (threads + 255) / 256, most = num_sms * 16L;
  return static_cast<unsigned>(want < 1 ? 1 : want < most ? want : most);
}

template <typename T, int GROUP, bool BACKWARD>
cudaError_t copy_group(const VocabArgs &a, int num_sms, cudaStream_t s) {
  const unsigned blocks = blocks_of((a.rows + 127L) * GROUP, num_sms);
  if (a.rows <= 256 * kRowItems) {
    HostTrace t("vocab_rows_gather", s);
    // every block reads all labels: no more blocks than give each a few rows
    vocab_rows_gather_kernel<T, GROUP, BACKWARD><<<blocks < 2u * num_sms ? blocks : 2u * num_sms, 256, 0, s>>>(a);
    return cudaGetLastError();
  }
  {
    HostTrace t("vocab_rows", s);
    vocab_rows_kernel<BACKWARD><<<1, kRowThreads, 0, s>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  HostTrace t("vocab_gather", s);
  return launch_early(vocab_gather_kernel<T, GROUP, BACKWARD>, blocks, 256, s, a);
}

template <typename T, bool BACKWARD>
cudaError_t copy_rows(const VocabArgs &a, int num_sms, cudaStream_t s) {
  return a.ld_xs >= kWideRow ? copy_group<T, 256, BACKWARD>(a, num_sms, s) : copy_group<T, 32, BACKWARD>(a, num_sms, s);
}

cudaError_t copies(const VocabArgs &a, bool backward, int num_sms, cudaStream_t s) {
  if (a.pad_w) {
    HostTrace t("vocab_pad", s);
    vocab_pad_kernel<<<blocks_of(static_cast<long>(a.V) * (a.ld_ws_w >> 3), num_sms), 256, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.dtype == MOE_ELEM_BF16)
    return backward ? copy_rows<__nv_bfloat16, true>(a, num_sms, s) : copy_rows<__nv_bfloat16, false>(a, num_sms, s);
  return backward ? copy_rows<__half, true>(a, num_sms, s) : copy_rows<__half, false>(a, num_sms, s);
}

}  // namespace

cudaError_t launch_vocab_forward(const VocabArgs &a, int num_sms, cudaStream_t s) {
  if (a.rows == 0) return cudaMemsetAsync(a.status, 0, 256, s);
  cudaError_t e = copies(a, false, num_sms, s);
  if (e == cudaSuccess) e = launch_vocab_tc(a, VOCAB_LOSS, s);
  if (e != cudaSuccess) return e;
  HostTrace t("vocab_loss", s);
  if (a.rows <= 8 * num_sms && a.parts > 64) return launch_early(vocab_loss_kernel<256>, a.rows, 256, s, a);
  return launch_early(vocab_loss_kernel<32>, blocks_of(static_cast<long>(a.rows) * 32, num_sms), 256, s, a);
}

cudaError_t launch_vocab_backward(const VocabArgs &given, int num_sms, cudaStream_t s) {
  VocabArgs a = given;
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    e = copies(a, true, num_sms, s);
  } else {
    e = cudaMemsetAsync(a.status, 0, 256, s);  // status and count: no rows
  }
  for (a.v0 = 0; a.v0 < a.V && e == cudaSuccess; a.v0 += a.width) {
    a.wp = a.V - a.v0 < a.width ? a.V - a.v0 : a.width;
    if (a.rows > 0) e = launch_vocab_tc(a, VOCAB_DZ, s);
    if (e == cudaSuccess && a.dx && a.rows > 0) e = launch_vocab_tc(a, VOCAB_DX, s);
    if (e == cudaSuccess && a.dw) e = launch_vocab_tc(a, VOCAB_DW, s);
  }
  if (e != cudaSuccess || !a.dx || a.rows == 0) return e;
  const bool vec = (reinterpret_cast<uintptr_t>(a.dx) & 15) == 0 && a.ld_dx % 8 == 0 && a.d % 8 == 0;
  HostTrace t("vocab_dx", s);
  const unsigned blocks = blocks_of(static_cast<long>(a.rows) * ((a.d + 7) / 8), num_sms);
  return a.dtype == MOE_ELEM_BF16 ? launch_early(vocab_dx_kernel<__nv_bfloat16>, blocks, 256, s, a, vec)
                                  : launch_early(vocab_dx_kernel<__half>, blocks, 256, s, a, vec);
}

}  // namespace moe
