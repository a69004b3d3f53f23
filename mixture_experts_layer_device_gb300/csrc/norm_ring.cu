// Norm kernels for many rows (the mathematics stands in norm.cu).  A row is cut
// at the 16-byte boundaries of memory, and each chunk belongs to a fixed thread,
// which copies its own chunks of the rows to come into its own places in shared
// memory (cp.async) and waits for its own copies only: rows are in flight while
// others are summed, without a producer, and without registers for what has not
// arrived.  The thread's column weights stay in its registers as fp32 (a channel
// gate multiplied into w_post); two columns share an instruction (f32x2).
//
// Rows whose width or stride is no multiple of 16 bytes (EDGES) start anywhere in
// a chunk.  The grid is a multiple of the pattern's period, so all rows of a
// block start at the same place in their first chunk and a thread's columns stay
// the same; chunks at a row's ends hold a neighbour's values, which are taken
// out before the sums, and are stored element by element.
#include "gemm_common.cuh"
#include "kernels.h"
#include "norm.cuh"

namespace moe {

namespace {

// Rows that share the forward's two barriers: two where two blocks fit an SM (16384 x
// 4096: 88 us, 98 with three), three where one takes most of its registers and shared
// memory (16384 x 7168: 150 us, 171 with two; x 5120: 121 and 138).
__host__ __device__ constexpr int fwd_rows(int threads) { return threads > 288 && threads <= 512 ? 3 : 2; }
constexpr int kRingSmem = 232448 - 2048;

// 16-byte chunks of a row per thread: 16 columns of a 2-byte type, 8 of fp32 (in
// the backward, 8 columns of bf16 cost 302 us where 16 cost 238 at 16384 x 6144:
// what a warp does once per row then weighs twice).
constexpr int kChunks = 2;

// 16 bytes to shared memory, of which the first `bytes` are read and the rest zeros.
MOE_DEV void copy16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
MOE_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most n of this thread's groups are in flight.
MOE_DEV void copy_wait(int n) {
  if (n <= 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else asm volatile("cp.async.wait_group 3;" ::: "memory");
}
MOE_DEV uint4 lds16(uint32_t at) {
  uint4 q;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at));
  return q;
}
MOE_DEV void sts_zero16(uint32_t at) { asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0)); }
// Under a predicate, without a branch: 16 bytes to shared memory, and st_stream.
MOE_DEV void sts16_if(bool on, uint32_t at, const uint4 &q) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n @p st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n}\n" ::"r"(at),
               "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w), "r"(static_cast<uint32_t>(on))
               : "memory");
}
MOE_DEV void st_stream_if(bool on, void *p, const uint4 &q) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n @p st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};\n}\n" ::"l"(p),
               "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w), "r"(static_cast<uint32_t>(on)));
}

// One thread's columns of a row: chunk i covers the VEC columns from at(i) on, of
// which those in [lo(i), hi(i)) exist.  `shift`: how far into a chunk the rows start.
template <typename T, bool EDGES>
struct Columns {
  static constexpr int VEC = Elem<T>::VEC;
  int c0, step, d;
  uint32_t head[4];  // bits of the first chunk that are the row's
  MOE_DEV Columns(int cols, int shift) : c0(threadIdx.x * VEC - (EDGES ? shift : 0)), step(blockDim.x * VEC), d(cols) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int out = lo(0) * static_cast<int>(sizeof(T)) - 4 * k;  // bytes of the word in front of the row
      head[k] = out >= 4 ? 0u : (out == 2 ? 0xffff0000u : 0xffffffffu);
    }
  }
  MOE_DEV int at(int i) const { return c0 + i * step; }
  MOE_DEV bool has(int i) const { return at(i) < d; }
  MOE_DEV int lo(int i) const { return EDGES && at(i) < 0 ? -at(i) : 0; }
  MOE_DEV int hi(int i) const { return EDGES && d - at(i) < VEC ? d - at(i) : VEC; }
  MOE_DEV bool whole(int i) const { return EDGES ? at(i) >= 0 && at(i) + VEC <= d : has(i); }
  // bytes of the chunk that lie in the row or before it
  MOE_DEV int bytes(int i) const { return EDGES ? hi(i) * static_cast<int>(sizeof(T)) : 16; }

  // what the copy left in shared memory: it filled up with zeros behind the row's end; in
  // front of its start (thread 0's first chunk) stands the end of the row before
  MOE_DEV void unpack(int i, uint4 q, f32x2 *p) const {
    if (EDGES && i == 0) {
      q.x &= head[0];
      q.y &= head[1];
      q.z &= head[2];
      q.w &= head[3];
    }
    unpack_pairs<T>(q, p);
  }
  // at column at(0) + i * step of the row that `row0` points at column at(0) of
  MOE_DEV void store(int i, T *row0, const f32x2 *p) const {
    T *dst = row0 + i * step;
    const uint4 q = pack_pairs<T>(p);
    if (whole(i)) {
      st_stream(dst, q);
    } else {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        if (k < lo(i) || k >= hi(i)) continue;
        if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t *>(dst)[k] = w[k];
        else reinterpret_cast<uint16_t *>(dst)[k] = static_cast<uint16_t>(w[k / 2] >> (k % 2 * 16));
      }
    }
  }
  // The same without a branch; a chunk that the row has only a part of goes to parts[0]
  // (its first) or parts[1] (its last), for put_part after a barrier.
  MOE_DEV void store_or_keep(bool on, int i, T *row0, const f32x2 *p, uint4 *parts) const {
    const uint4 q = pack_pairs<T>(p);
    st_stream_if(on && whole(i), row0 + i * step, q);
    if (EDGES) sts16_if(has(i) && !whole(i), smem_u32(parts + (at(i) < 0 ? 0 : 1)), q);
  }
  MOE_DEV void weights(int i, const void *w, float *v) const {
    const T *p = static_cast<const T *>(w);
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = p && has(i) && k >= lo(i) && k < hi(i) ? Elem<T>::to(p[at(i) + k]) : 1.f;
  }
};

// fp32 weights of this thread's columns: w_pre, and w_post times a channel gate.
template <typename T, bool EDGES>
MOE_DEV void own_weights(const NormArgs &a, const Columns<T, EDGES> &col, f32x2 (*wp)[Elem<T>::VEC / 2],
                         f32x2 (*w)[Elem<T>::VEC / 2]) {
  constexpr int VEC = Elem<T>::VEC;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    float u[VEC], v[VEC], g[VEC];
    col.weights(i, a.w_pre, u);
    col.weights(i, a.w_post, v);
    col.weights(i, a.gate == MOE_GATE_CHANNEL ? a.g : nullptr, g);
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) {
      wp[i][k] = f2_of(u[2 * k], u[2 * k + 1]);
      w[i][k] = f2_of(v[2 * k] * g[2 * k], v[2 * k + 1] * g[2 * k + 1]);
    }
  }
}

// Element j of a row's first and last chunk (Columns::store_or_keep) to the row; j < 2 VEC.
template <typename T>
MOE_DEV void put_part(T *row, int d, int shift, int j, const uint4 *parts) {
  constexpr int VEC = Elem<T>::VEC;
  const int last = j / VEC, k = j % VEC, c = last ? (d + shift) / VEC * VEC - shift + k : k - shift;
  if (last ? c < d : c >= 0 && shift > 0) row[c] = reinterpret_cast<const T *>(parts + last)[k];
}

// ---------------------------------------------------------------- forward
// fwd_rows() rows at a time (a grid apart): their sums share the barriers.  Shared
// memory: [stage][row][x, f, full gate][chunk][thread] of 16 bytes.
template <typename T, bool FULL, bool EDGES, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 288 ? 2 : 1) norm_fwd_ring_kernel(const NormArgs a, int stages) {
  constexpr int P = Elem<T>::VEC / 2, NT = FULL ? 3 : 2, R = fwd_rows(THREADS), SUMS = R > 2 ? 4 : R;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[2][SUMS][kMaxWarps];
  // as in the backward, the rows' first and last chunks leave after a barrier (8000 x 2883
  // with a full gate: 48 us, 53 from the threads that have them), but where registers are
  // short (16384 x 4095: 128 us so, 113)
  constexpr bool KEEP = EDGES && THREADS <= 256;
  __shared__ __align__(16) uint4 parts[2][R][2][2];  // [turn][row][z, h][first, last]
  int part_turn = 0;
  const int shift = row_shift<T>(a.ld_x, blockIdx.x);
  const Columns<T, EDGES> col(a.d, shift);
  const uint32_t place = 16 * blockDim.x, stage_bytes = R * NT * kChunks * place;
  const uint32_t base = smem_u32(smem) + 16 * threadIdx.x;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const bool post = (a.flags & MOE_NORM_POST) != 0, pre = (a.flags & MOE_NORM_PRE) != 0;
  const long G = gridDim.x, step = G * R;
  auto fetch = [&](long row, uint32_t at) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const long q = row + r * G;
      if (q < a.rows) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          if (col.has(i)) {
            const uint32_t p = at + (r * NT * kChunks + i) * place;
            const int n = col.bytes(i);
            copy16(p, static_cast<const T *>(a.x) + q * a.ld_x + col.at(i), n);
            if (a.f) copy16(p + kChunks * place, static_cast<const T *>(a.f) + q * a.ld_f + col.at(i), n);
            if (FULL) copy16(p + 2 * kChunks * place, static_cast<const T *>(a.g) + q * a.ld_g + col.at(i), n);
          }
      }
    }
    copy_commit();
  };
  auto put = [&](int i, T *row0, const f32x2 *p, uint4 *parts_of) {
    if (KEEP) col.store_or_keep(true, i, row0, p, parts_of);
    else col.store(i, row0, p);
  };
  long row = blockIdx.x;
  for (int k = 0; k + 1 < stages; ++k) fetch(row + k * step, base + k * stage_bytes);
  f32x2 wp[kChunks][P], w[kChunks][P];
  own_weights<T, EDGES>(a, col, wp, w);
  const f32x2 alpha = f2_both(a.alpha);
  int turn = 0, stage = 0, ahead = stages - 1;
  for (; row < a.rows; row += step) {
    float rg[R];
#pragma unroll
    for (int r = 0; r < R; ++r) rg[r] = row + r * G < a.rows ? row_gate_of<T>(a, row + r * G) : 1.f;
    fetch(row + (stages - 1) * step, base + ahead * stage_bytes);
    copy_wait(stages - 1);
    const uint32_t at = base + stage * stage_bytes;
    uint4 fq[R][kChunks];
    float ss[SUMS];
    for (int r = R; r < SUMS; ++r) ss[r] = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f32x2 sum = 0;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        fq[r][i] = make_uint4(0, 0, 0, 0);
        if (a.f && col.has(i)) fq[r][i] = lds16(at + ((r * NT + 1) * kChunks + i) * place);
        f32x2 v[P];
        col.unpack(i, fq[r][i], v);
#pragma unroll
        for (int k = 0; k < P; ++k) sum = f2_fma(v[k], v[k], sum);
      }
      ss[r] = f2_sum(sum);
    }
    if (post) {
      row_sum<false, SUMS>(ss, red, turn);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float rp = rsqrtf(ss[r] * inv_d + a.eps);
        if (threadIdx.x == 0 && a.r_post && row + r * G < a.rows) a.r_post[row + r * G] = rp;
        rg[r] *= rp;
      }
    }
    f32x2 z[R][kChunks][P];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const f32x2 rr = f2_both(rg[r]);
      f32x2 sum = 0;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
#pragma unroll
        for (int k = 0; k < P; ++k) z[r][i][k] = 0;
        if (col.has(i)) {
          f32x2 v[P], g[P];
          col.unpack(i, lds16(at + (r * NT * kChunks + i) * place), z[r][i]);
          col.unpack(i, fq[r][i], v);
          if (FULL) col.unpack(i, lds16(at + ((r * NT + 2) * kChunks + i) * place), g);
#pragma unroll
          for (int k = 0; k < P; ++k) {
            v[k] = f2_mul(v[k], rr);
            if (FULL) v[k] = f2_mul(v[k], g[k]);
            z[r][i][k] = f2_fma(v[k], w[i][k], f2_mul(alpha, z[r][i][k]));
            sum = f2_fma(z[r][i][k], z[r][i][k], sum);
          }
          if (a.z && row + r * G < a.rows)
            put(i, static_cast<T *>(a.z) + (row + r * G) * a.ld_z + col.at(0), z[r][i], parts[part_turn][r][0]);
        }
      }
      ss[r] = f2_sum(sum);
    }
    if (pre) {
      row_sum<false, SUMS>(ss, red, turn);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (row + r * G >= a.rows) break;
        const float rp = rsqrtf(ss[r] * inv_d + a.eps);
        const f32x2 rr = f2_both(rp);
        if (threadIdx.x == 0 && a.r_pre) a.r_pre[row + r * G] = rp;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          if (col.has(i)) {
#pragma unroll
            for (int k = 0; k < P; ++k) z[r][i][k] = f2_mul(z[r][i][k], f2_mul(rr, wp[i][k]));
            put(i, static_cast<T *>(a.h) + (row + r * G) * a.ld_h + col.at(0), z[r][i], parts[part_turn][r][1]);
          }
      }
    }
    if (KEEP) {
      constexpr int N = 2 * Elem<T>::VEC;
      __syncthreads();
      for (int j = threadIdx.x; j < R * 2 * N; j += blockDim.x) {
        const int r = j / (2 * N), t = j / N % 2;
        T *out = static_cast<T *>(t ? a.h : a.z);
        if (out && row + r * G < a.rows)
          put_part(out + (row + r * G) * (t ? a.ld_h : a.ld_z), a.d, shift, j % N, parts[part_turn][r][t]);
      }
      part_turn ^= 1;
    }
    if (++stage == stages) stage = 0;
    if (++ahead == stages) ahead = 0;
  }
}

// ---------------------------------------------------------------- backward
// Shared memory: [stage][dz, dh, z, f, full gate][chunk][thread] of 16 bytes.
// The loops are those of add_sums and elem_out (norm.cuh), two columns at once.
// One step sums row i + 1 and finishes row i, so the barrier and the joining of
// the sums have the other row's work beside them.  POST by kernel: asked per element,
// whether f is in df costs 232 us where this takes 194 (16384 x 6144).
template <typename T, bool POST, bool FULL, bool EDGES, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 2 : 1) norm_bwd_ring_kernel(const NormArgs a, int stages) {
  pdl_trigger();
  constexpr int VEC = Elem<T>::VEC, P = VEC / 2, NT = FULL ? 5 : 4;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[2][4][kMaxWarps];
  long row = blockIdx.x;
  const int shift = row_shift<T>(a.ld_z, row);
  const Columns<T, EDGES> col(a.d, shift);
  const uint32_t place = 16 * blockDim.x, stage_bytes = NT * kChunks * place;
  const uint32_t base = smem_u32(smem) + 16 * threadIdx.x;
  const float inv_d = 1.f / static_cast<float>(a.d);
  const bool pre = (a.flags & MOE_NORM_PRE) != 0;
  const long step = gridDim.x;
  // this thread's first column of the next row to fetch (NULL: not there)
  const T *src[NT];
  long hop[NT];
  auto source = [&](int t, const void *p, long ld) {
    src[t] = p ? static_cast<const T *>(p) + row * ld + col.at(0) : nullptr;
    hop[t] = step * ld;
  };
  source(0, a.dz, a.ld_z);
  source(1, pre ? a.dh : nullptr, a.ld_h);
  source(2, pre ? a.zin : nullptr, a.ld_z);
  source(3, a.f, a.ld_f);
  if (FULL) source(NT - 1, a.g, a.ld_g);
  long coming = row;
  auto fetch = [&](uint32_t at) {
    if (coming < a.rows) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (src[t]) {
#pragma unroll
          for (int i = 0; i < kChunks; ++i)
            if (col.has(i)) copy16(at + (t * kChunks + i) * place, src[t] + i * col.step, col.bytes(i));
          src[t] += hop[t];
        }
    }
    coming += step;
    copy_commit();
  };
  // a tensor or chunk that is not there reads as zeros
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if (!src[t] || !col.has(i))
        for (int k = 0; k < stages; ++k) sts_zero16(base + k * stage_bytes + (t * kChunks + i) * place);
  auto take = [&](uint32_t at, int t, int i, f32x2 *p) { col.unpack(i, lds16(at + (t * kChunks + i) * place), p); };
  for (int k = 0; k + 1 < stages; ++k) fetch(base + k * stage_bytes);
  f32x2 wp[kChunks][P], w[kChunks][P], acc0[kChunks][P], acc1[kChunks][P];
  own_weights<T, EDGES>(a, col, wp, w);
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
#pragma unroll
    for (int k = 0; k < P; ++k) acc0[i][k] = acc1[i][k] = 0;
  T *dx = a.dx ? static_cast<T *>(a.dx) + row * a.ld_x + col.at(0) : nullptr;
  T *df = a.df ? static_cast<T *>(a.df) + row * a.ld_f + col.at(0) : nullptr;
  T *dg = FULL && a.dg ? static_cast<T *>(a.dg) + row * a.ld_g + col.at(0) : nullptr;
  const f32x2 alpha = f2_both(a.alpha);
  auto sums = [&](uint32_t at, float (*out)[kMaxWarps]) {
    f32x2 s2[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      f32x2 dz[P], dh[P], z[P], f[P], g[P];
      take(at, 0, i, dz);
      take(at, 1, i, dh);
      take(at, 2, i, z);
      take(at, 3, i, f);
      if (FULL) take(at, NT - 1, i, g);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const f32x2 u = f2_mul(dh[k], wp[i][k]);
        f32x2 v = f2_mul(f[k], w[i][k]);
        if (FULL) v = f2_mul(v, g[k]);
        s2[0] = f2_fma(u, z[k], s2[0]);
        s2[1] = f2_fma(dz[k], v, s2[1]);
        s2[2] = f2_fma(u, v, s2[2]);
        s2[3] = f2_fma(z[k], v, s2[3]);
      }
    }
    float s[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = f2_sum(s2[k]);
    block_sums_put<4>(s, out);
  };
  // Straight-line code: the chunks' arithmetic then runs side by side.  The chunks that
  // the row has a part of, its first and last, go to shared memory and leave after the
  // row's barrier, an element per thread (from the one thread that has them, 8000 x 2883:
  // 118 us where this took 97; 93 now).
  __shared__ __align__(16) uint4 parts[2][3][2];  // [turn][dx, df, dg][first, last]
  int turn = 0;
  auto put_parts = [&](int of, long r) {
    for (int j = threadIdx.x; j < 3 * 2 * VEC; j += blockDim.x) {
      const int t = j / (2 * VEC);
      T *out = static_cast<T *>(t == 0 ? a.dx : (t == 1 ? a.df : (FULL ? a.dg : nullptr)));
      if (out) put_part(out + r * (t == 0 ? a.ld_x : (t == 1 ? a.ld_f : a.ld_g)), a.d, shift, j % (2 * VEC), parts[of][t]);
    }
  };
  int stage = 0, ahead = stages - 1;
  RowIn in = {}, next = {};
  if (row < a.rows) {
    in = row_in<T>(a, row);
    copy_wait(stages - 2);
    sums(base, red[0]);
  }
  __syncthreads();
  for (; row < a.rows; row += step) {
    const bool more = row + step < a.rows;
    if (EDGES && row > blockIdx.x) put_parts(turn ^ 1, row - step);
    if (more) next = row_in<T>(a, row + step);
    fetch(base + ahead * stage_bytes);
    copy_wait(stages - 2);
    const int after = stage + 1 == stages ? 0 : stage + 1;
    if (more) sums(base + after * stage_bytes, red[turn ^ 1]);
    float s[4];
    block_sums_get<4>(s, red[turn]);
    const RowTerms t = row_terms<T>(a, POST, row, in, s, inv_d, threadIdx.x == 0);
    const f32x2 rp = f2_both(t.rp), c1 = f2_both(-t.c1), a1 = f2_both(t.a1), c2 = f2_both(-t.c2);
    const uint32_t at = base + stage * stage_bytes;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      f32x2 dz[P], dh[P], z[P], f[P], g[P], o[P];
      take(at, 0, i, dz);
      take(at, 1, i, dh);
      take(at, 2, i, z);
      take(at, 3, i, f);
      if (FULL) take(at, NT - 1, i, g);
#pragma unroll
      for (int k = 0; k < P; ++k) {
        const f32x2 y = f2_mul(rp, z[k]);
        const f32x2 tt = f2_fma(rp, f2_mul(dh[k], wp[i][k]), f2_fma(c1, y, dz[k]));
        acc0[i][k] = f2_fma(dh[k], y, acc0[i][k]);
        const f32x2 nh = f2_mul(f[k], a1);
        f32x2 tg = tt, tw = f2_mul(tt, w[i][k]);
        if (FULL) {
          o[k] = f2_mul(tw, nh);
          tg = f2_mul(tg, g[k]);
          tw = f2_mul(tw, g[k]);
        }
        acc1[i][k] = f2_fma(tg, nh, acc1[i][k]);
        dz[k] = f2_mul(alpha, tt);
        f[k] = f2_fma(a1, tw, POST ? f2_mul(c2, nh) : 0);
      }
      col.store_or_keep(dx, i, dx, dz, parts[turn][0]);
      col.store_or_keep(df, i, df, f, parts[turn][1]);
      if (FULL) col.store_or_keep(dg, i, dg, o, parts[turn][2]);
    }
    if (dx) dx += step * a.ld_x;
    if (df) df += step * a.ld_f;
    if (FULL && dg) dg += step * a.ld_g;
    in = next;
    turn ^= 1;
    stage = after;
    if (++ahead == stages) ahead = 0;
    __syncthreads();
  }
  if (EDGES && row > blockIdx.x) put_parts(turn ^ 1, row - step);
  if (a.part) {
    // by place in the chunks: columns that are not the row's hold zeros and are not read
    const long ld_p = norm_part_row(a.d);
    float *p = a.part + blockIdx.x * 2 * ld_p + threadIdx.x * VEC;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if (col.has(i)) {
        float u[VEC], v[VEC];
#pragma unroll
        for (int k = 0; k < P; ++k) {
          f2_split(acc0[i][k], u[2 * k], u[2 * k + 1]);
          f2_split(acc1[i][k], v[2 * k], v[2 * k + 1]);
        }
        put_sums<VEC>(p + i * col.step, u);
        put_sums<VEC>(p + ld_p + i * col.step, v);
      }
  }
}

// Threads, stages and shared memory of a call; stages 0: the kernels do not take it.
struct RingShape {
  int threads, stages;
  size_t smem;
  bool edges;
};
RingShape ring_shape(const NormArgs &a, bool backward) {
  RingShape r = {};
  const int esz = elem_bytes(a.dtype), vec = 16 / esz;
  // every row of the call has to start at the same place in its first chunk
  const long m = a.ld_z % vec;
  auto fits = [&](const void *p, long ld) { return !p || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % vec == m); };
  if (!fits(a.x, a.ld_x) || !fits(a.f, a.ld_f) || !fits(a.z, a.ld_z) || !fits(a.h, a.ld_h) || !fits(a.dz, a.ld_z) ||
      !fits(a.zin, a.ld_z) || !fits(a.dh, a.ld_h) || !fits(a.dx, a.ld_x) || !fits(a.df, a.ld_f))
    return r;
  if (a.gate == MOE_GATE_FULL && (!fits(a.g, a.ld_g) || !fits(a.dg, a.ld_g))) return r;
  r.edges = m != 0 || a.d % vec != 0;
  const int nt = (backward ? 4 : 2) + (a.gate == MOE_GATE_FULL ? 1 : 0);
  const int per = kChunks * vec;
  r.threads = ((a.d + (m ? vec - 1 : 0) + per - 1) / per + 31) / 32 * 32;
  if (r.threads > (backward ? 512 : 1024)) return r;
  const size_t stage = static_cast<size_t>(r.threads) * kChunks * 16 * nt * (backward ? 1 : fwd_rows(r.threads));
  // short rows: three stages and more blocks
  for (int s = r.threads <= (backward ? 256 : 288) ? 3 : 4; s >= 2; --s)
    if (stage * s <= kRingSmem) {
      r.stages = s;
      r.smem = stage * s;
      break;
    }
  return r;
}

template <typename K>
cudaError_t ring_launch(K kernel, const NormArgs &a, const RingShape &r, int num_sms, int most_blocks, int *slots,
                        int (&memo)[33][64], cudaStream_t s) {
  // the shape follows from the threads and the full gate, so one answer per kernel and block size
  const int per_sm = per_device_memo(memo[r.threads >> 5], [&]() {
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem) != cudaSuccess) return 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, r.threads, r.smem) == cudaSuccess ? n : 0;
  });
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  long grid = static_cast<long>(num_sms) * per_sm;
  if (grid > a.rows) grid = a.rows;
  if (grid > most_blocks) grid = most_blocks;
  grid = grid / 8 * 8;  // the period of the rows' places in a chunk divides 8; more rows than SMs come here
  *slots = static_cast<int>(grid);
  kernel<<<static_cast<int>(grid), r.threads, r.smem, s>>>(a, r.stages);
  return cudaGetLastError();
}

template <typename T, bool FULL, bool EDGES, int THREADS>
cudaError_t fwd_shape(const NormArgs &a, const RingShape &r, int num_sms, cudaStream_t s) {
  static int memo[33][64] = {};
  int slots;
  return ring_launch(norm_fwd_ring_kernel<T, FULL, EDGES, THREADS>, a, r, num_sms, 1 << 30, &slots, memo, s);
}
template <typename T, bool POST, bool FULL, bool EDGES, int THREADS>
cudaError_t bwd_shape(const NormArgs &a, const RingShape &r, int num_sms, int *slots, cudaStream_t s) {
  static int memo[33][64] = {};
  return ring_launch(norm_bwd_ring_kernel<T, POST, FULL, EDGES, THREADS>, a, r, num_sms, norm_max_blocks(a.d), slots, memo, s);
}

// Block sizes by the registers that they leave a thread: up to 256 threads two
// blocks (128), the forward's 288 too (96; 16384 x 4608: 97 us, 134 with one block),
// the backward's 384 one (168), 512 (128), 1024 (64).
template <typename T, bool FULL, bool EDGES>
cudaError_t fwd_block(const NormArgs &a, const RingShape &r, int num_sms, cudaStream_t s) {
  if (r.threads <= 256) return fwd_shape<T, FULL, EDGES, 256>(a, r, num_sms, s);
  if (r.threads <= 288) return fwd_shape<T, FULL, EDGES, 288>(a, r, num_sms, s);
  if (r.threads <= 512) return fwd_shape<T, FULL, EDGES, 512>(a, r, num_sms, s);
  return fwd_shape<T, FULL, EDGES, 1024>(a, r, num_sms, s);
}
template <typename T, bool POST, bool FULL, bool EDGES>
cudaError_t bwd_block(const NormArgs &a, const RingShape &r, int num_sms, int *slots, cudaStream_t s) {
  if (r.threads <= 256) return bwd_shape<T, POST, FULL, EDGES, 256>(a, r, num_sms, slots, s);
  if (r.threads <= 384) return bwd_shape<T, POST, FULL, EDGES, 384>(a, r, num_sms, slots, s);
  return bwd_shape<T, POST, FULL, EDGES, 512>(a, r, num_sms, slots, s);
}

template <typename T>
cudaError_t fwd_type(const NormArgs &a, int num_sms, cudaStream_t s) {
  const RingShape r = ring_shape(a, false);
  if (a.gate == MOE_GATE_FULL)
    return r.edges ? fwd_block<T, true, true>(a, r, num_sms, s) : fwd_block<T, true, false>(a, r, num_sms, s);
  return r.edges ? fwd_block<T, false, true>(a, r, num_sms, s) : fwd_block<T, false, false>(a, r, num_sms, s);
}
template <typename T, bool POST>
cudaError_t bwd_gate(const NormArgs &a, int num_sms, int *slots, cudaStream_t s) {
  const RingShape r = ring_shape(a, true);
  if (a.gate == MOE_GATE_FULL)
    return r.edges ? bwd_block<T, POST, true, true>(a, r, num_sms, slots, s)
                   : bwd_block<T, POST, true, false>(a, r, num_sms, slots, s);
  return r.edges ? bwd_block<T, POST, false, true>(a, r, num_sms, slots, s)
                 : bwd_block<T, POST, false, false>(a, r, num_sms, slots, s);
}
template <typename T>
cudaError_t bwd_type(const NormArgs &a, int num_sms, int *slots, cudaStream_t s) {
  return (a.flags & MOE_NORM_POST) ? bwd_gate<T, true>(a, num_sms, slots, s) : bwd_gate<T, false>(a, num_sms, slots, s);
}

}  // namespace

bool norm_ring_fits(const NormArgs &a, bool backward) { return ring_shape(a, backward).stages > 0 && a.d > 256; }

cudaError_t launch_norm_fwd_ring(const NormArgs &a, int num_sms, cudaStream_t s) {
  switch (a.dtype) {
    case MOE_ELEM_BF16: return fwd_type<__nv_bfloat16>(a, num_sms, s);
    case MOE_ELEM_FP16: return fwd_type<__half>(a, num_sms, s);
    default: return fwd_type<float>(a, num_sms, s);
  }
}

cudaError_t launch_norm_bwd_ring(const NormArgs &a, int num_sms, int *slots, cudaStream_t s) {
  switch (a.dtype) {
    case MOE_ELEM_BF16: return bwd_type<__nv_bfloat16>(a, num_sms, slots, s);
    case MOE_ELEM_FP16: return bwd_type<__half>(a, num_sms, slots, s);
    default: return bwd_type<float>(a, num_sms, slots, s);
  }
}

}  // namespace moe
