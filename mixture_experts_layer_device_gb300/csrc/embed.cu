// Token embedding and its gradient.
//   out[t] = scale table[ids[t]];   dtable[v] = scale sum over ids[t] = v of dout[t]
// The gradient sorts the tokens by id (stable), so that the rows of one id lie
// next to each other in ascending token order, and cuts the sorted list into
// pieces.  A block sums a piece's runs in fp32; a run that lies
// inside its piece is final, one that crosses into others leaves a partial row,
// and a last pass joins the partial rows of such a run in order.  A frequent id
// is so spread over many blocks, and every sum has one fixed order.
//
// HBM bound: forward one row in, one out per token; backward one row in per
// token and the whole table out (or, accumulating, the rows that occur, twice).
#include "block.h"
#include "elem.cuh"
#include "gemm_common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kMaxPiece = 64;   // sorted tokens per block of the sums: 64, or 16 of few
__host__ __device__ inline int piece_of(long rows) { return rows > 8192 ? kMaxPiece : 16; }
constexpr int kSmallSort = 2048;  // up to here every token counts its rank
constexpr int kSortBlock = 256;   // threads of a radix block
constexpr int kSortItems = 2;     // keys per thread and block: the passes are short, so more blocks
constexpr int kSortChunk = kSortBlock * kSortItems;
constexpr int kMaxDigits = 1024;  // 10-bit digits at most

// Table row of token t, or V for an id outside the table.
MOE_DEV int key_of(const EmbedArgs &a, long t) {
  if (a.ids64) {
    const long long v = static_cast<const long long *>(a.ids)[t];
    return (v >= 0 && v < a.V) ? static_cast<int>(v) : a.V;
  }
  const int v = static_cast<const int *>(a.ids)[t];
  return (v >= 0 && v < a.V) ? v : a.V;
}

// ---------------------------------------------------------------- forward
// A warp takes 32 x UN chunks (16 bytes each) of one row at a time, all its
// loads in flight before the first store.
template <typename T, int VEC, int UN>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const EmbedArgs a, int spans) {
  const int lane = threadIdx.x & 31;
  const long warps = static_cast<long>(gridDim.x) * (blockDim.x >> 5);
  const long total = static_cast<long>(a.rows) * spans;
  for (long u = static_cast<long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); u < total; u += warps) {
    const long row = u / spans;
    const int c0 = static_cast<int>(u - row * spans) * 32 * UN * VEC + lane * VEC;
    const int key = key_of(a, row);
    T *dst = static_cast<T *>(a.out) + row * a.ld_o;
    const T *src = static_cast<const T *>(a.table) + static_cast<long>(key) * a.ld_t;
    if constexpr (VEC > 1) {
      uint4 q[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        q[i] = make_uint4(0, 0, 0, 0);
        if (key < a.V && c0 + i * 32 * VEC < a.d) q[i] = __ldg(reinterpret_cast<const uint4 *>(src + c0 + i * 32 * VEC));
      }
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        if (c0 + i * 32 * VEC >= a.d) continue;
        float v[VEC];
        Elem<T>::unpack(q[i], v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = key < a.V ? v[k] * a.scale : 0.f;
        st_stream(dst + c0 + i * 32 * VEC, Elem<T>::pack(v));
      }
    } else {
      T q[UN];
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        q[i] = Elem<T>::from(0.f);
        if (key < a.V && c0 + i * 32 < a.d) q[i] = src[c0 + i * 32];
      }
#pragma unroll
      for (int i = 0; i < UN; ++i)
        if (c0 + i * 32 < a.d) dst[c0 + i * 32] = Elem<T>::from(key < a.V ? Elem<T>::to(q[i]) * a.scale : 0.f);
    }
  }
}

// ---------------------------------------------------------------- fill
// Zeros for the table rows of [from, to) that no token points to, a warp per row,
// in the sums' launch.  (Filling slices beside the sort's launches too, which
// leave the memory idle, measured 247 us where this is 250: not kept.)
struct Fill {
  const uint8_t *used;
  uint8_t *table;
  long row_bytes, ld_bytes;
  int unit;  // bytes per store: 16, or an element of unaligned rows
  int from, to;
};
MOE_DEV void fill_rows(const Fill &f, long block, long blocks) {
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  for (long v = f.from + block * warps + (threadIdx.x >> 5); v < f.to; v += blocks * warps) {
    if (f.used[v]) continue;
    uint8_t *dst = f.table + v * f.ld_bytes;
    if (f.unit == 16) {
      for (long b = lane * 16; b < f.row_bytes; b += 512) st_stream(dst + b, make_uint4(0, 0, 0, 0));
    } else if (f.unit == 4) {
      for (long b = lane * 4; b < f.row_bytes; b += 128) *reinterpret_cast<uint32_t *>(dst + b) = 0;
    } else {
      for (long b = lane * 2; b < f.row_bytes; b += 64) *reinterpret_cast<uint16_t *>(dst + b) = 0;
    }
  }
}

// ---------------------------------------------------------------- sort
// Few tokens: a token's place is the number of tokens that come before it.
// One launch instead of a radix pass' three per digit; 2,048 comparisons a
// thread at most.  Also marks the table rows that occur.
constexpr int kRankBlock = 128;
__global__ void __launch_bounds__(kRankBlock) embed_rank_kernel(const EmbedArgs a, int *keys, int *pos, uint8_t *used) {
  pdl_trigger();
  __shared__ int sk[kSmallSort];
  for (int i = threadIdx.x; i < a.rows; i += kRankBlock) sk[i] = key_of(a, i);
  __syncthreads();
  const int t = blockIdx.x * kRankBlock + threadIdx.x;
  if (t >= a.rows) return;
  const int key = sk[t];
  int rank = 0;
#pragma unroll 8
  for (int i = 0; i < t; ++i) rank += sk[i] <= key;
#pragma unroll 8
  for (int i = t + 1; i < a.rows; ++i) rank += sk[i] < key;
  keys[rank] = key;
  pos[rank] = t;
  if (used && key < a.V) used[key] = 1;
}

// Up to 65,536 tokens: the whole radix sort in one launch of one cluster.  Each of
// its eight blocks holds a consecutive piece of the list in shared memory; a pass
// ranks the piece's keys (stable), adds up the digits' counts of all blocks
// through distributed shared memory, orders the piece by digit in place, and
// writes it out from there: neighbouring threads then mostly write neighbouring
// places of one block (written straight from the ranking, every lane's store
// goes somewhere else: 27 us where this takes 21, and the six launches of the
// larger sort 31, at 32768 tokens and 18-bit keys).
constexpr int kClusterBlocks = 8, kClusterThreads = 1024, kClusterItems = 8, kClusterDigits = 512;
constexpr int kClusterSort = kClusterBlocks * kClusterThreads * kClusterItems;

struct ClusterSmem {
  int2 list[2][kClusterThreads * kClusterItems];          // key, position
  uint16_t count[kClusterThreads / 32][kClusterDigits];  // per warp and digit: keys so far, then keys of the warps before
  int total[kClusterDigits];                              // this block's keys of a digit
  int base[kClusterDigits];                               // first place of this block's keys of a digit
  int start[kClusterDigits];                              // the same within the block
  int2 warp_sum[kClusterDigits / 32];
};
static_assert(sizeof(ClusterSmem) <= 232448, "shared memory");

MOE_DEV int ld_cluster(uint32_t at) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
MOE_DEV void st_cluster(uint32_t at, int2 v) {
  asm volatile("st.shared::cluster.v2.s32 [%0], {%1, %2};" ::"r"(at), "r"(v.x), "r"(v.y) : "memory");
}

__global__ void __cluster_dims__(kClusterBlocks, 1, 1) __launch_bounds__(kClusterThreads, 1)
    embed_cluster_sort_kernel(const EmbedArgs a, int items, int passes, int bits, int *keys_out, int *pos_out, uint8_t *used) {
  pdl_trigger();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  ClusterSmem &sm = *reinterpret_cast<ClusterSmem *>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, digits = 1 << bits;
  const uint32_t rank = cluster_rank();
  const int piece = kClusterThreads * items, first = static_cast<int>(rank) * piece;
  const int held = a.rows - first < piece ? (a.rows > first ? a.rows - first : 0) : piece;  // places of the piece in the list
  const int mine = warp * 32 * items + lane;  // a warp ranks 32 x items consecutive keys
  for (int i = 0; i < items; ++i) {
    const int at = mine + 32 * i;
    if (at < held) {
      const int key = key_of(a, first + at);
      if (used && key < a.V) used[key] = 1;
      sm.list[0][at] = make_int2(key, first + at);
    }
  }
  for (int p = 0; p < passes; ++p) {
    const int in = p & 1, shift = p * bits;
    for (int i = threadIdx.x; i < (kClusterThreads / 32) * kClusterDigits / 8; i += kClusterThreads)
      reinterpret_cast<uint4 *>(sm.count)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    int2 kv[kClusterItems];
    int local[kClusterItems];
#pragma unroll
    for (int i = 0; i < kClusterItems; ++i) {
      if (i >= items) break;
      const bool has = mine + 32 * i < held;
      int dg = digits;  // places past the end: a group of their own
      if (has) {
        kv[i] = sm.list[in][mine + 32 * i];
        dg = (kv[i].x >> shift) & (digits - 1);
      }
      const unsigned same = __match_any_sync(0xffffffffu, dg);
      const int before = __popc(same & ((1u << lane) - 1));
      if (has) local[i] = sm.count[warp][dg] + before;
      __syncwarp();
      if (has && before == 0) sm.count[warp][dg] += static_cast<uint16_t>(__popc(same));
      __syncwarp();
    }
    __syncthreads();
    int own = 0, all = 0, before = 0;
    const bool digit = static_cast<int>(threadIdx.x) < digits;
    if (digit) {
#pragma unroll 8
      for (int w = 0; w < kClusterThreads / 32; ++w) {
        const int n = sm.count[w][threadIdx.x];
        sm.count[w][threadIdx.x] = static_cast<uint16_t>(own);
        own += n;
      }
      sm.total[threadIdx.x] = own;
    }
    cluster_sync();
    // places of this block's keys: those of smaller digits anywhere, and of the same digit in the blocks before
    if (digit) {
      const uint32_t at = smem_u32(&sm.total[threadIdx.x]);
      int n[kClusterBlocks];
#pragma unroll
      for (int c = 0; c < kClusterBlocks; ++c) n[c] = ld_cluster(peer_smem(at, c));
#pragma unroll
      for (int c = 0; c < kClusterBlocks; ++c) {
        all += n[c];
        if (c < static_cast<int>(rank)) before += n[c];
      }
    }
    int inc = all, inc_own = own;
    if (threadIdx.x < kClusterDigits) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, inc, o), m = __shfl_up_sync(0xffffffffu, inc_own, o);
        if (lane >= o) {
          inc += n;
          inc_own += m;
        }
      }
      if (lane == 31) sm.warp_sum[warp] = make_int2(inc, inc_own);
    }
    __syncthreads();
    if (threadIdx.x < kClusterDigits) {  // whole warps, whatever the number of digits
      const int2 v = lane < warp ? sm.warp_sum[lane] : make_int2(0, 0);  // warp <= 15: the warps before
      sm.base[threadIdx.x] = __reduce_add_sync(0xffffffffu, v.x) + before + inc - all;
      sm.start[threadIdx.x] = __reduce_add_sync(0xffffffffu, v.y) + inc_own - own;
    }
    __syncthreads();
    // the piece in order of digits, where the pass read it from
#pragma unroll
    for (int i = 0; i < kClusterItems; ++i) {
      if (i >= items || mine + 32 * i >= held) break;
      const int dg = (kv[i].x >> shift) & (digits - 1);
      sm.list[in][sm.start[dg] + sm.count[warp][dg] + local[i]] = kv[i];
    }
    __syncthreads();
    for (int at = threadIdx.x; at < held; at += kClusterThreads) {
      const int2 v = sm.list[in][at];
      const int dg = (v.x >> shift) & (digits - 1), to = sm.base[dg] + at - sm.start[dg];
      if (p + 1 == passes) {
        keys_out[to] = v.x;
        pos_out[to] = v.y;
      } else {
        const int block = to / piece;
        st_cluster(peer_smem(smem_u32(&sm.list[in ^ 1][to - block * piece]), block), v);
      }
    }
    cluster_sync();  // the keys have arrived; no block leaves or reuses its counts while another reads them
  }
}

// One digit of the least-significant-digit radix sort: histogram per block,
// prefix over the blocks of every digit, stable scatter.  `keys` NULL: the ids.
__global__ void __launch_bounds__(kSortBlock) embed_hist_kernel(const EmbedArgs a, const int *keys, int shift,
                                                                int digits, int *hist, uint8_t *used) {
  __shared__ int h[kMaxDigits];
  for (int i = threadIdx.x; i < digits; i += kSortBlock) h[i] = 0;
  __syncthreads();
  const long base = static_cast<long>(blockIdx.x) * kSortChunk;
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const long i = base + k * kSortBlock + threadIdx.x;
    if (i < a.rows) {
      const int key = keys ? keys[i] : key_of(a, i);
      atomicAdd(&h[(key >> shift) & (digits - 1)], 1);
      if (used && key < a.V) used[key] = 1;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < digits; i += kSortBlock) hist[static_cast<long>(i) * gridDim.x + blockIdx.x] = h[i];
}

// Exclusive prefix of one digit's block counts (a warp per digit), its total.
__global__ void __launch_bounds__(256) embed_scan_kernel(int *hist, int blocks, int digits, int *total) {
  const int digit = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (digit >= digits) return;
  int *h = hist + static_cast<long>(digit) * blocks;
  int run = 0;
  for (int b = 0; b < blocks; b += 32) {
    const int v = b + lane < blocks ? h[b + lane] : 0;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    if (b + lane < blocks) h[b + lane] = run + inc - v;
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) total[digit] = run;
}

// Block offset of `digits` totals: exclusive prefix into out[] by one warp.
MOE_DEV void warp_prefix(const int *total, int digits, int *out) {
  const int lane = threadIdx.x & 31;
  int run = 0;
  for (int i = 0; i < digits; i += 32) {
    const int v = i + lane < digits ? total[i + lane] : 0;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    if (i + lane < digits) out[i + lane] = run + inc - v;
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
}

__global__ void __launch_bounds__(kSortBlock) embed_scatter_kernel(const EmbedArgs a, const int *keys, const int *pos,
                                                                   int shift, int digits, const int *hist,
                                                                   const int *total, int *keys_out, int *pos_out) {
  pdl_trigger();
  // next[w][digit]: where warp w's next key of a digit goes
  extern __shared__ int next[];
  __shared__ int base[kMaxDigits];
  constexpr int W = kSortBlock / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < W * digits; i += kSortBlock) next[i] = 0;
  if (warp == 0) warp_prefix(total, digits, base);
  __syncthreads();
  // a warp owns kSortItems consecutive groups of 32 keys
  const long first = static_cast<long>(blockIdx.x) * kSortChunk + warp * 32 * kSortItems + lane;
  int key[kSortItems], ps[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const long i = first + k * 32;
    key[k] = -1;
    if (i < a.rows) {
      key[k] = keys ? keys[i] : key_of(a, i);
      ps[k] = pos ? pos[i] : static_cast<int>(i);
      atomicAdd(&next[warp * digits + ((key[k] >> shift) & (digits - 1))], 1);
    }
  }
  __syncthreads();
  for (int dg = threadIdx.x; dg < digits; dg += kSortBlock) {
    int at = base[dg] + hist[static_cast<long>(dg) * gridDim.x + blockIdx.x];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int n = next[w * digits + dg];
      next[w * digits + dg] = at;
      at += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const bool in = key[k] >= 0;
    const int dg = in ? (key[k] >> shift) & (digits - 1) : digits;  // keys out of range form their own group
    const unsigned same = __match_any_sync(0xffffffffu, dg);
    const int before = __popc(same & ((1u << lane) - 1));
    int at = 0;
    if (in) at = next[warp * digits + dg] + before;
    __syncwarp();
    if (in && before == 0) next[warp * digits + dg] += __popc(same);
    __syncwarp();
    if (in) {
      keys_out[at] = key[k];
      pos_out[at] = ps[k];
    }
  }
}

// ---------------------------------------------------------------- sums
// Writes (or adds) a finished fp32 sum of VEC columns to the table.
template <typename G, int VEC>
MOE_DEV void put_grad(const EmbedArgs &a, int key, int c, const float *acc) {
  G *dst = static_cast<G *>(a.dtable) + static_cast<long>(key) * a.ld_t + c;
  float v[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    v[k] = acc[k] * a.scale;
    if (a.accumulate) v[k] += Elem<G>::to(dst[k]);
  }
  if constexpr (VEC == Elem<G>::VEC) {
    st_stream(dst, Elem<G>::pack(v));
  } else if constexpr (VEC == 2 * Elem<G>::VEC) {
    st_stream(dst, Elem<G>::pack(v));
    st_stream(dst + VEC / 2, Elem<G>::pack(v + VEC / 2));
  } else if constexpr (2 * VEC == Elem<G>::VEC) {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(Elem<G>::pack2(v[0], v[1]), Elem<G>::pack2(v[2], v[3]));
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) dst[k] = Elem<G>::from(v[k]);
  }
}

// Blocks below pieces * slabs: the rows of one piece x 128 threads' columns.
// part[2 p] takes the run that comes in from piece p - 1, part[2 p + 1] the one
// that starts here and goes on in piece p + 1; such runs enter the list cross
// (16 bytes each from the second on: first piece, last piece, table row; their
// number in the first word; the order does not matter, each is joined by
// itself).  The other blocks write the rows of zeros beside it.
template <typename T, typename G, int VEC>
__global__ void __launch_bounds__(128) embed_sum_kernel(const EmbedArgs a, const int *keys, const int *pos, float *part,
                                                        int *cross, int pieces, int slabs, const Fill fill) {
  __shared__ int sk[kMaxPiece], sp[kMaxPiece];
  pdl_wait();
  pdl_trigger();
  const long work = static_cast<long>(pieces) * slabs;
  if (blockIdx.x >= work) {
    fill_rows(fill, blockIdx.x - work, gridDim.x - work);
    return;
  }
  const int slab = blockIdx.x % slabs;
  const int piece = blockIdx.x / slabs;
  const int len = piece_of(a.rows), first = piece * len;
  const int n = a.rows - first < len ? a.rows - first : len;
  if (threadIdx.x < n) {
    sk[threadIdx.x] = keys[first + threadIdx.x];
    sp[threadIdx.x] = pos[first + threadIdx.x];
  }
  const int before = first > 0 ? keys[first - 1] : -1;
  const int after = first + n < a.rows ? keys[first + n] : -1;
  __syncthreads();
  if (slab == 0 && threadIdx.x == 0) {
    const int last = sk[n - 1];
    if (last < a.V && after == last && !(before == last && sk[0] == last)) {
      // the last piece that the run reaches: the first token of a piece has its key
      int lo = piece + 1, hi = pieces - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (keys[mid * len] == last) lo = mid;
        else hi = mid - 1;
      }
      reinterpret_cast<int4 *>(cross)[1 + atomicAdd(cross, 1)] = make_int4(piece, lo, last, 0);
    }
  }
  const int c = (slab * 128 + threadIdx.x) * VEC;
  if (c >= a.d) return;
  float acc[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
  constexpr int U = VEC > 1 ? 8 : 16;
  int run = 0;  // first token of the current run
  for (int j0 = 0; j0 < n; j0 += U) {
    uint4 q[U];
    T q1[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j0 + u < n && sk[j0 + u] < a.V) {
        const T *p = static_cast<const T *>(a.dout) + static_cast<long>(sp[j0 + u]) * a.ld_o + c;
        if constexpr (VEC > 1) q[u] = ld_stream(p);
        else q1[u] = *p;
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u;
      if (j >= n) break;
      const int key = sk[j];
      if (key >= a.V) break;  // padding sorts last
      float v[VEC];
      if constexpr (VEC > 1) Elem<T>::unpack(q[u], v);
      else v[0] = Elem<T>::to(q1[u]);
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[k] += v[k];
      const int nextkey = j + 1 < n ? sk[j + 1] : after;
      const bool ends = j + 1 == n || nextkey != key;
      if (ends) {
        const bool came = run == 0 && before == key, goes = nextkey == key;
        if (!came && !goes) {
          put_grad<G, VEC>(a, key, c, acc);
        } else {
          float *p = part + (static_cast<long>(piece) * 2 + (came ? 0 : 1)) * a.d + c;
#pragma unroll
          for (int k = 0; k < VEC; ++k) p[k] = acc[k];
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
        run = j + 1;
      }
    }
  }
}

// Joins the runs that cross pieces: 256 x VEC columns of one run per block, its
// partial rows in order.
template <typename G, int VEC>
__global__ void __launch_bounds__(256) embed_join_kernel(const EmbedArgs a, const float *part, const int *cross, int slabs) {
  pdl_wait();
  const long total = static_cast<long>(cross[0]) * slabs;
  for (long u = blockIdx.x; u < total; u += gridDim.x) {
    const int4 run = reinterpret_cast<const int4 *>(cross)[1 + u / slabs];
    const int c = (static_cast<int>(u % slabs) * 256 + threadIdx.x) * VEC;
    if (c >= a.d) continue;
    // the starting piece's second row, then the first rows of those after it
    float acc[VEC];
    auto load = [&](long row, float *v) {
      const float *p = part + row * a.d + c;
      if constexpr (VEC == 4) {
        const float4 q = *reinterpret_cast<const float4 *>(p);
        v[0] = q.x;
        v[1] = q.y;
        v[2] = q.z;
        v[3] = q.w;
      } else {
        v[0] = *p;
      }
    };
    load(2L * run.x + 1, acc);
    int i = run.x + 1;
    for (; i + 7 <= run.y; i += 8) {
      float v[8][VEC];
#pragma unroll
      for (int k = 0; k < 8; ++k) load(2L * (i + k), v[k]);
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] += v[k][j];
    }
    for (; i <= run.y; ++i) {
      float v[VEC];
      load(2L * i, v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] += v[j];
    }
    put_grad<G, VEC>(a, run.z, c, acc);
  }
}

// Bits of the keys 0 .. V.
int key_bits(long V) {
  int bits = 1;
  while ((1L << bits) <= V) ++bits;
  return bits;
}

struct EmbedWs {
  size_t keys[2], pos[2], hist, total, cross, used, part, bytes;
};

EmbedWs ws_layout(int rows, long V, int d) {
  EmbedWs w;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += (n + 255) / 256 * 256;
    return o;
  };
  const size_t T = rows, blocks = (T + kSortChunk - 1) / kSortChunk, pieces = (T + piece_of(rows) - 1) / piece_of(rows);
  for (int i = 0; i < 2; ++i) {
    w.keys[i] = take(T * 4);
    w.pos[i] = take(T * 4);
  }
  w.hist = take(blocks * kMaxDigits * 4);
  w.total = take(kMaxDigits * 4);
  w.used = take(V);
  w.cross = take((pieces + 1) * 16);
  w.part = take(pieces * 2 * d * 4);
  w.bytes = at;
  return w;
}

bool vec16(const void *p, long ld, int esz) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * esz) % 16 == 0;
}

template <typename T>
cudaError_t fwd_type(const EmbedArgs &a, cudaStream_t s) {
  const int e = sizeof(T);
  const bool vec = vec16(a.table, a.ld_t, e) && vec16(a.out, a.ld_o, e) && (static_cast<long>(a.d) * e) % 16 == 0;
  constexpr int UN = 4;
  const int cols = 32 * UN * (vec ? Elem<T>::VEC : 1);
  const int spans = (a.d + cols - 1) / cols;
  const long blocks = (static_cast<long>(a.rows) * spans + 7) / 8;
  const int grid = static_cast<int>(blocks < 152 * 64 ? blocks : 152 * 64);
  if (vec) embed_fwd_kernel<T, Elem<T>::VEC, UN><<<grid, 256, 0, s>>>(a, spans);
  else embed_fwd_kernel<T, 1, UN><<<grid, 256, 0, s>>>(a, spans);
  return cudaGetLastError();
}

template <typename T, typename G>
cudaError_t sums(const EmbedArgs &a, const int *keys, const int *pos, float *part, int *cross, const Fill &fill,
                 int num_sms, cudaStream_t s) {
  const int pieces = (a.rows + piece_of(a.rows) - 1) / piece_of(a.rows);
  const bool vec = vec16(a.dout, a.ld_o, sizeof(T)) && vec16(a.dtable, a.ld_t, sizeof(G)) &&
                   a.d % Elem<T>::VEC == 0 && a.d % Elem<G>::VEC == 0;
  const int cols = 128 * (vec ? Elem<T>::VEC : 1), slabs = (a.d + cols - 1) / cols;
  // a fill block's four warps take a table row each, so many rows a block
  const long rows_left = (static_cast<long>(fill.to) - fill.from + 3) / 4, most = num_sms * 32L;
  const long grid = static_cast<long>(pieces) * slabs + (rows_left < most ? rows_left : most);
  if (grid > 2147483647L) return cudaErrorInvalidConfiguration;
  if (grid) {
    HostTrace t("embed_sum", s);
    const auto kernel = vec ? embed_sum_kernel<T, G, Elem<T>::VEC> : embed_sum_kernel<T, G, 1>;
    cudaError_t e;
    if (a.rows > 0) {  // behind the sort
      e = launch_early(kernel, static_cast<unsigned>(grid), 128, s, a, keys, pos, part, cross, pieces, slabs, fill);
    } else {
      kernel<<<static_cast<unsigned>(grid), 128, 0, s>>>(a, keys, pos, part, cross, pieces, slabs, fill);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
  }
  if (pieces > 1) {
    HostTrace t("embed_join", s);
    const int join_cols = 256 * (vec ? 4 : 1), join_slabs = (a.d + join_cols - 1) / join_cols;
    const long want = static_cast<long>(pieces) * join_slabs;
    const unsigned blocks = static_cast<unsigned>(want < num_sms * 8L ? want : num_sms * 8L);
    return launch_early(vec ? embed_join_kernel<G, 4> : embed_join_kernel<G, 1>, blocks, 256, s, a, part, cross, join_slabs);
  }
  return cudaSuccess;
}

}  // namespace

size_t embed_workspace(int rows, long V, int d) { return ws_layout(rows, V, d).bytes; }

cudaError_t launch_embed_forward(const EmbedArgs &a, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  HostTrace t("embed_forward", s);
  switch (a.dtype) {
    case MOE_ELEM_BF16: return fwd_type<__nv_bfloat16>(a, s);
    case MOE_ELEM_FP16: return fwd_type<__half>(a, s);
    default: return fwd_type<float>(a, s);
  }
}

cudaError_t launch_embed_backward(const EmbedArgs &a, int num_sms, cudaStream_t s) {
  const EmbedWs w = ws_layout(a.rows, a.V, a.d);
  int *keys[2], *pos[2];
  for (int i = 0; i < 2; ++i) {
    keys[i] = reinterpret_cast<int *>(a.ws + w.keys[i]);
    pos[i] = reinterpret_cast<int *>(a.ws + w.pos[i]);
  }
  uint8_t *used = a.accumulate ? nullptr : a.ws + w.used;
  float *part = reinterpret_cast<float *>(a.ws + w.part);
  int *cross = reinterpret_cast<int *>(a.ws + w.cross);
  // the flags of the table rows and the number of crossing runs lie together
  cudaError_t e = used ? cudaMemsetAsync(used, 0, w.cross + 4 - w.used, s) : cudaMemsetAsync(cross, 0, 4, s);
  if (e != cudaSuccess) return e;
  const long gsz = elem_bytes(a.grad_dtype);
  Fill fill = {used, static_cast<uint8_t *>(a.dtable), a.d * gsz, a.ld_t * gsz, static_cast<int>(gsz), 0,
               a.accumulate ? 0 : a.V};
  if (vec16(a.dtable, a.ld_t, static_cast<int>(gsz)) && fill.row_bytes % 16 == 0) fill.unit = 16;
  int at = 0;
  if (a.rows > 0 && a.rows <= kSmallSort) {
    HostTrace t("embed_rank", s);
    embed_rank_kernel<<<(a.rows + kRankBlock - 1) / kRankBlock, kRankBlock, 0, s>>>(a, keys[0], pos[0], used);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  } else if (a.rows > 0 && a.rows <= kClusterSort) {
    HostTrace t("embed_sort", s);
    const int bits = key_bits(a.V), passes = (bits + 8) / 9, per = (bits + passes - 1) / passes;
    const int items = (a.rows + kClusterBlocks * kClusterThreads - 1) / (kClusterBlocks * kClusterThreads);
    static int memo[64] = {};
    if (per_device_memo(memo, []() {
          return cudaFuncSetAttribute(embed_cluster_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(sizeof(ClusterSmem))) == cudaSuccess
                     ? 1
                     : 0;
        }) <= 0)
      return cudaErrorInvalidConfiguration;
    embed_cluster_sort_kernel<<<kClusterBlocks, kClusterThreads, sizeof(ClusterSmem), s>>>(a, items, passes, per, keys[0], pos[0],
                                                                                         used);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  } else if (a.rows > 0) {
    const int bits = key_bits(a.V);
    const int passes = (bits + 9) / 10;
    const int per = (bits + passes - 1) / passes;
    const int blocks = (a.rows + kSortChunk - 1) / kSortChunk;
    int *hist = reinterpret_cast<int *>(a.ws + w.hist), *total = reinterpret_cast<int *>(a.ws + w.total);
    const int digits = 1 << per;
    for (int p = 0; p < passes; ++p) {
      const int *kin = p ? keys[at] : nullptr, *pin = p ? pos[at] : nullptr;
      const int to = p ? at ^ 1 : 0;
      HostTrace t("embed_sort", s);
      embed_hist_kernel<<<blocks, kSortBlock, 0, s>>>(a, kin, p * per, digits, hist, p ? nullptr : used);
      embed_scan_kernel<<<(digits + 7) / 8, 256, 0, s>>>(hist, blocks, digits, total);
      embed_scatter_kernel<<<blocks, kSortBlock, static_cast<size_t>(digits) * (kSortBlock / 32) * 4, s>>>(
          a, kin, pin, p * per, digits, hist, total, keys[to], pos[to]);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      at = to;
    }
  }
  const int *k = keys[at], *ps = pos[at];
  const bool wide = a.grad_dtype == MOE_ELEM_FP32;
  switch (a.dtype) {
    case MOE_ELEM_BF16:
      return wide ? sums<__nv_bfloat16, float>(a, k, ps, part, cross, fill, num_sms, s)
                  : sums<__nv_bfloat16, __nv_bfloat16>(a, k, ps, part, cross, fill, num_sms, s);
    case MOE_ELEM_FP16:
      return wide ? sums<__half, float>(a, k, ps, part, cross, fill, num_sms, s)
                  : sums<__half, __half>(a, k, ps, part, cross, fill, num_sms, s);
    default: return sums<float, float>(a, k, ps, part, cross, fill, num_sms, s);
  }
}

}  // namespace moe
