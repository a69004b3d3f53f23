// The global norm of many gradients, and their clipping:
//   norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + eps)),  out = c g
//
// Two launches: blocks leave sums of squares, then one warp of each block of the next
// launch adds those up in the same order (a few kilobytes from L2) and the block scales.
// (The whole block adding, and each of its threads taking root and quotient, cost 17 us on
// the slow 64-bit pipes of a call that scales nothing.)  The tensors' addresses and lengths
// travel as launch parameters, so nothing is copied to the device and a captured graph
// keeps them.
//
// Bound by memory: the norm reads everything once.  Clipping reads it again (from the end
// backwards, for what L2 might still hold, it took as long: 3e8 bf16 into fp32 290 us either
// way); in place and below the limit (c = 1) it reads and writes nothing.
//
// Sums: a thread squares up to 64 elements in fp32 and adds that to a 64-bit
// sum.  Where fp32 overflows or its squares sink below the normal range, the
// same elements are squared again in 64 bits.
#include "block.h"
#include "elem.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kGradThreads = 256;
// 16-byte pieces per thread and chunk.  Chunks of 32 KB, blocks taking them in turns: 5.64 GB
// 816 us, 0.6 GB 109 us; of 16 KB with six blocks per SM 821 and 125; a block's chunks next
// to one another 851 and 124.
constexpr int kVecs = 8;
constexpr int kChunkVecs = kGradThreads * kVecs;
constexpr int kBlocksPerSm = 4;

// The tensors of one launch: their first elements, lengths and types, and the
// first chunk of each.  A chunk is kChunkVecs aligned 16-byte pieces; a tensor's
// first and last piece may be cut.
template <int MOST>
struct GradTable {
  int n, chunks;
  const uint8_t *data[MOST];
  uint8_t *out[MOST];
  int64_t count[MOST];
  int first[MOST + 1];
  uint8_t type[MOST], out_type[MOST];
};
// The smaller table where it holds them: a launch carries all of it (three tensors: 4.6 us of
// host time for the norm's two launches, 7.6 with the larger one).
constexpr int kFewTensors = 64, kManyTensors = 1024;
static_assert(sizeof(GradTable<kManyTensors>) + 64 <= 32764, "launch parameters");

// The tensor of chunk c, not before `lo` nor behind `hi`.
template <int MOST>
MOE_DEV int tensor_of_chunk(const GradTable<MOST> &t, int c, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The elements of a chunk that one thread takes, as raw 16-byte pieces; absent ones
// are zeros.  Elements in front of the tensor or behind it are not read.
template <typename T>
struct Piece {
  static constexpr int VEC = Elem<T>::VEC;
  const T *base;    // the aligned piece in which the tensor starts
  int64_t lead;     // elements in front of the tensor in it
  int64_t end;      // lead + count
  MOE_DEV Piece(const uint8_t *data, int64_t count) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(data);
    base = reinterpret_cast<const T *>(p & ~static_cast<uintptr_t>(15));
    lead = static_cast<int64_t>((p & 15) / sizeof(T));
    end = lead + count;
  }
  MOE_DEV bool whole(int64_t v) const { return v * VEC >= lead && v * VEC + VEC <= end; }
  MOE_DEV uint4 load(int64_t v) const {
    if (whole(v)) return ld_stream(base + v * VEC);
    union {
      uint4 q;
      T e[VEC];
    } u;
    u.q = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int64_t i = v * VEC + k;
      if (i >= lead && i < end) u.e[k] = base[i];
    }
    return u.q;
  }
};

// Sum of the squares of kVecs pieces in 64 bits.
template <typename T>
MOE_DEV double squares(const uint4 (&q)[kVecs]) {
  constexpr int VEC = Elem<T>::VEC;
  float s0 = 0.f, s1 = 0.f;
  uint32_t any = 0;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    float v[VEC];
    Elem<T>::unpack(q[j], v);
#pragma unroll
    for (int k = 0; k < VEC; k += 2) {
      s0 = fmaf(v[k], v[k], s0);
      s1 = fmaf(v[k + 1], v[k + 1], s1);
    }
    any |= q[j].x | q[j].y | q[j].z | q[j].w;
  }
  const float s = s0 + s1;
  // from 2^-110 on, 64 squares that are each off by half of fp32's smallest step do not count
  const uint32_t magnitude = sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu;
  if ((s >= 7.7e-34f && s <= 3.0e38f) || (any & magnitude) == 0) return s;
  double d = 0.0;
#pragma unroll 1
  for (int j = 0; j < kVecs; ++j) {
    float v[VEC];
    uint4 p = q[0];
#pragma unroll
    for (int i = 1; i < kVecs; ++i)
      if (i == j) p = q[i];
    Elem<T>::unpack(p, v);
#pragma unroll
    for (int k = 0; k < VEC; ++k) d = fma(static_cast<double>(v[k]), static_cast<double>(v[k]), d);
  }
  return d;
}

template <typename T>
MOE_DEV double chunk_squares(const uint8_t *data, int64_t count, int local) {
  const Piece<T> p(data, count);
  const int64_t v0 = static_cast<int64_t>(local) * kChunkVecs + threadIdx.x;
  uint4 q[kVecs];
  if (v0 * Piece<T>::VEC >= p.end) return 0.0;
#pragma unroll
  for (int j = 0; j < kVecs; ++j) q[j] = p.load(v0 + j * kGradThreads);
  return squares<T>(q);
}

// A block's sum of its threads' values, in a fixed order; valid in thread 0.
MOE_DEV double block_sum(double v) {
  __shared__ double part[kGradThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kGradThreads / 32; ++w) s += part[w];
  return s;
}

template <int MOST>
__global__ void __launch_bounds__(kGradThreads, kBlocksPerSm) grad_squares_kernel(const __grid_constant__ GradTable<MOST> t,
                                                                                  double *part) {
  pdl_trigger();
  double sum = 0.0;
  int i = 0;
  for (int c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    if (t.first[i + 1] <= c) i = tensor_of_chunk(t, c, i + 1, t.n - 1);
    const int local = c - t.first[i];
    if (t.type[i] == MOE_ELEM_BF16) sum += chunk_squares<__nv_bfloat16>(t.data[i], t.count[i], local);
    else if (t.type[i] == MOE_ELEM_FP16) sum += chunk_squares<__half>(t.data[i], t.count[i], local);
    else sum += chunk_squares<float>(t.data[i], t.count[i], local);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The norm from all blocks' sums, by one warp.
MOE_DEV double norm_of(const double *part, int n) {
  double v[4] = {0.0, 0.0, 0.0, 0.0};
  for (int i = threadIdx.x; i < n; i += 128)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + 32 * k < n) v[k] += part[i + 32 * k];
  double s = (v[0] + v[1]) + (v[2] + v[3]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return sqrt(s);
}

__global__ void __launch_bounds__(32) grad_norm_kernel(const double *part, int n, float *norm) {
  pdl_wait();
  const double v = norm_of(part, n);
  if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

MOE_DEV void st_stream_32(void *p, const float *f) {
  asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
               "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}

// One thread's pieces of a chunk, times c, to `out`.
template <typename T, typename O>
MOE_DEV void chunk_scale(const uint8_t *data, uint8_t *out, int64_t count, int local, float c) {
  constexpr int VEC = Elem<T>::VEC;
  const Piece<T> p(data, count);
  O *o = reinterpret_cast<O *>(out) - p.lead;  // the place of piece 0's first element
  // a piece leaves in one store: 16 bytes, or 32 as fp32 from 16-bit elements
  constexpr int OUT = VEC * static_cast<int>(sizeof(O));
  const bool vec = (reinterpret_cast<uintptr_t>(o) & (OUT - 1)) == 0;
  const int64_t v0 = static_cast<int64_t>(local) * kChunkVecs + threadIdx.x;
  if (v0 * VEC >= p.end) return;
  uint4 q[kVecs];
#pragma unroll
  for (int j = 0; j < kVecs; ++j) q[j] = p.load(v0 + j * kGradThreads);
#pragma unroll
  for (int j = 0; j < kVecs; ++j) {
    const int64_t v = v0 + j * kGradThreads;
    float f[VEC];
    Elem<T>::unpack(q[j], f);
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] *= c;
    if (vec && p.whole(v)) {
      if constexpr (OUT == 32) st_stream_32(o + v * VEC, f);
      else st_stream(o + v * VEC, Elem<O>::pack(f));
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const int64_t i = v * VEC + k;
        if (i >= p.lead && i < p.end) o[i] = Elem<O>::from(f[k]);
      }
    }
  }
}

template <typename T>
MOE_DEV void chunk_scale_to(const uint8_t *data, uint8_t *out, int out_type, int64_t count, int local, float c) {
  if (out_type == MOE_ELEM_FP32) chunk_scale<T, float>(data, out, count, local, c);
  else chunk_scale<T, T>(data, out, count, local, c);
}

template <int MOST>
__global__ void __launch_bounds__(kGradThreads, kBlocksPerSm) grad_scale_kernel(const __grid_constant__ GradTable<MOST> t,
                                                                     const double *part, int n, double max_norm,
                                                                     double eps, bool in_place, float *norm) {
  __shared__ float factor;
  pdl_wait();
  if (threadIdx.x < 32) {
    const double v = norm_of(part, n);
    if (threadIdx.x == 0) {
      if (blockIdx.x == 0) *norm = static_cast<float>(v);
      // no limit: an infinite norm scales nothing either (inf / inf is NaN)
      const double r = isinf(max_norm) && isinf(v) ? 1.0 : max_norm / (v + eps);
      factor = r >= 1.0 ? 1.f : static_cast<float>(r);  // NaN stays
    }
  }
  __syncthreads();
  const float c = factor;
  if (c == 1.f && in_place) return;
  int i = 0;
  for (int chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
    if (t.first[i + 1] <= chunk) i = tensor_of_chunk(t, chunk, i + 1, t.n - 1);
    const int local = chunk - t.first[i];
    if (c == 1.f && t.out[i] == t.data[i]) continue;
    if (t.type[i] == MOE_ELEM_BF16) chunk_scale_to<__nv_bfloat16>(t.data[i], t.out[i], t.out_type[i], t.count[i], local, c);
    else if (t.type[i] == MOE_ELEM_FP16) chunk_scale_to<__half>(t.data[i], t.out[i], t.out_type[i], t.count[i], local, c);
    else chunk_scale_to<float>(t.data[i], t.out[i], t.out_type[i], t.count[i], local, c);
  }
}

long tensor_chunks(const GradTensors &g, int i) {
  const int64_t e = elem_bytes(g.dtypes[i]);
  const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(g.data[i]) & 15) / e;
  const int64_t vecs = (lead + g.counts[i] + 16 / e - 1) / (16 / e);
  return static_cast<long>((vecs + kChunkVecs - 1) / kChunkVecs);
}

// The next launch's tensors, from `at` on: as many as the table holds.  Empty ones are
// left out.  (Their chunks, 32 KB each, are counted in 32 bits.)
template <int MOST>
int fill_table(GradTable<MOST> *t, const GradTensors &g, int at) {
  t->n = 0;
  long chunks = 0;
  for (; at < g.n && t->n < MOST; ++at) {
    if (g.counts[at] == 0) continue;
    const long more = tensor_chunks(g, at);
    const int i = t->n++;
    t->data[i] = static_cast<const uint8_t *>(g.data[at]);
    t->out[i] = g.outs ? static_cast<uint8_t *>(g.outs[at]) : nullptr;
    t->count[i] = g.counts[at];
    t->type[i] = static_cast<uint8_t>(g.dtypes[at]);
    t->out_type[i] = static_cast<uint8_t>(g.outs ? g.out_dtypes[at] : 0);
    t->first[i] = static_cast<int>(chunks);
    chunks += more;
  }
  t->chunks = static_cast<int>(chunks);
  t->first[t->n] = t->chunks;
  return at;
}

// The workspace has room for so many sums per launch.
constexpr int kMostBlocks = kBlocksPerSm * 152;
int grid_of(int chunks, int num_sms) {
  const int most = num_sms * kBlocksPerSm < kMostBlocks ? num_sms * kBlocksPerSm : kMostBlocks;
  return chunks < most ? chunks : most;
}

template <int MOST>
cudaError_t grads(const GradTensors &g, bool clip, double max_norm, double eps, float *norm, double *part, int num_sms,
                  cudaStream_t s) {
  GradTable<MOST> t;
  int sums = 0;
  for (int at = 0; at < g.n;) {
    at = fill_table(&t, g, at);
    if (t.chunks == 0) break;
    HostTrace trace("grad_squares", s);
    const int grid = grid_of(t.chunks, num_sms);
    grad_squares_kernel<MOST><<<grid, kGradThreads, 0, s>>>(t, part + sums);
    sums += grid;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (!clip || sums == 0) {
    HostTrace trace("grad_norm", s);
    return launch_early(grad_norm_kernel, 1, 32, s, static_cast<const double *>(part), sums, norm);
  }
  bool in_place = true;
  for (int i = 0; i < g.n; ++i) in_place &= g.outs[i] == g.data[i];
  for (int at = 0; at < g.n;) {
    at = g.n > MOST ? fill_table(&t, g, at) : g.n;  // one table: it is still there
    if (t.chunks == 0) break;
    HostTrace trace("grad_scale", s);
    e = launch_early(grad_scale_kernel<MOST>, grid_of(t.chunks, num_sms), kGradThreads, s, t,
                     static_cast<const double *>(part), sums, max_norm, eps, in_place, norm);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_workspace(int n) { return (static_cast<size_t>(n) / kManyTensors + 1) * kMostBlocks * sizeof(double); }

cudaError_t launch_grads(const GradTensors &g, bool clip, double max_norm, double eps, float *norm, void *ws, int num_sms,
                         cudaStream_t s) {
  double *part = static_cast<double *>(ws);
  return g.n <= kFewTensors ? grads<kFewTensors>(g, clip, max_norm, eps, norm, part, num_sms, s)
                            : grads<kManyTensors>(g, clip, max_norm, eps, norm, part, num_sms, s);
}

}  // namespace moe
