// Internal launchers of the operators around the layer (ragged grouped
// products, block norms, token embedding).  All launches are asynchronous on
// the given stream and return the launch error.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// ---------------------------------------------------------------- host services (api.cu)
// The current device's SM count after checking that it is an sm_103 part and
// that the tensor-map encoder is there: MOE_OK or a moe_status.
int host_device(int *num_sms);
// A tiled tensor map, 128-byte swizzle, zero fill out of bounds.
bool host_encode_map(CUtensorMap *m, int elem, const void *base, int rank, const uint64_t *dims,
                     const uint64_t *strides_bytes, const uint32_t *box);
// Brackets a launch with the trace's events when tracing is on (moe_trace_enable).
struct HostTrace {
  int slot;
  cudaStream_t s;
  HostTrace(const char *name, cudaStream_t stream);
  ~HostTrace();
};

// A launch that may begin while the kernel in front on the stream, which has to call
// pdl_trigger(), still runs: its blocks take their places and stop at pdl_wait() until
// that kernel has ended.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------- grouped products
// The three directions are one matrix product per expert, out[m, n] (+)= sum_k a[m, k]
// b[n, k], with the expert's rows on m (forward, dgrad) or on k (wgrad).  The plain kernel
// addresses both operands by two strides; the tensor-core kernel has the tokens on its
// instruction's N side and reads each operand in the major in which it lies.
enum GroupedDir { GROUPED_FWD = 0, GROUPED_DGRAD = 1, GROUPED_WGRAD = 2, GROUPED_GATED = 3 };

struct GroupedArgs {
  int E, N, K;
  int rows;
  int dtype, out_dtype;  // moe_elem; out_dtype of y / dw (dx has dtype)
  int accumulate;
  long ld_x, ld_y, ld_w, ld_e;
  long in_x, in_y;     // tensor-core path: row strides of the inputs x and dy (padded copies have their own)
  const int *offsets;  // [E + 1]
  const void *x, *w, *dy;
  void *y, *dx, *dw;
  // gated forward: N = 2 m rows of w, the gate's and the up projection's; y (may be NULL) keeps both
  // products, h [rows, m] = act(gate) up
  void *h;
  long ld_h;
  int act;  // moe_act
  bool vec_h, by_16;  // tensor-core path: h's rows are whole 16-byte pieces; m is a multiple of 16
  bool zeroed;   // weight gradient: launch_grouped_zero writes the experts without rows
  bool chained;  // tensor-core path: starts before the launch in front has ended (dgrad and wgrad of one call)
  bool vec_out;  // tensor-core path: the output's rows are whole 16-byte pieces
  int *status;   // workspace status word
  int most;      // tensor-core path: tokens of a tile at most
  int *tiles;    // workspace: the plan's tile table (3 E + 3 ints)
  int *order;    // workspace: the experts by descending rows, and how many have any (weight gradient)
  uint8_t *maps; // workspace: 2 E tensor maps of 128 bytes (weight gradient)
};

// The first launch of a call writes the status word (bad offsets) and zeroes the
// output rows of no expert: the plan does it for the plain kernel, whose tile
// table (first tile of `tile_rows` rows of every expert) it also makes, and for
// the tensor-core kernel with more experts than its shared memory holds
// (tile_rows 0: grouped.cuh's table); otherwise the kernels do it themselves.
cudaError_t launch_grouped_plan(const GroupedArgs &g, int tile_rows, void *out, int out_elem, int out_cols,
                                long ld_out, cudaStream_t s);
// Any size, stride and alignment; `first`: with the plan in front.
cudaError_t launch_grouped_plain(const GroupedArgs &g, int dir, bool first, cudaStream_t s);
// The gated forward for any size, stride and alignment, with its plans in front.
cudaError_t launch_gated_plain(const GroupedArgs &g, cudaStream_t s);
// Forward of a few rows (no plan needed): 16-byte aligned rows of x and w.
cudaError_t launch_grouped_few(const GroupedArgs &g, cudaStream_t s);
cudaError_t launch_gated_few(const GroupedArgs &g, cudaStream_t s);
// Puts the experts in order (g.order) for launch_grouped_zero; the tensor-core
// path's own launch does it there.
cudaError_t launch_grouped_order(const GroupedArgs &g, cudaStream_t s);
// Zeros for the weight gradients of experts without rows, right behind the launch
// that has put the experts in order.
cudaError_t launch_grouped_zero(const GroupedArgs &g, int num_sms, cudaStream_t s);
// dst [n rows of `cols`, stride ld_dst >= cols] = src with its row stride, zeros
// beyond cols; `experts`: rows of w (N per expert, ld_e apart), experts without
// rows left out.  2-byte elements.
cudaError_t launch_grouped_pad(const GroupedArgs &g, const void *src, long rows, int cols, long ld, bool experts,
                               void *dst, long ld_dst, cudaStream_t s);
// Tensor-core path: the operands' pointers and row strides multiples of 16 bytes.
cudaError_t launch_grouped_tc(const GroupedArgs &g, int dir, int num_sms, cudaStream_t s);
// Both products of a backward on it.
cudaError_t launch_grouped_tc_pair(GroupedArgs dgrad, GroupedArgs wgrad, int num_sms, cudaStream_t s);

// The gated products' backward in front of its two products: [dg | du] from dh and [g | u].
struct GatedArgs {
  int rows, m, dtype, act;
  long ld_h, ld_gu, ld_dgu;
  const void *dh, *gu;
  void *dgu;
};
cudaError_t launch_gated_slope(const GatedArgs &a, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------- block norms
struct NormArgs {
  int rows, d, dtype, flags, gate;
  float alpha, eps;
  long ld_x, ld_f, ld_z, ld_h, ld_g;
  const void *x, *f, *g, *w_post, *w_pre;
  void *z, *h;
  float *r_post, *r_pre;
  // backward
  const void *dz, *dh, *zin;
  const float *r_post_in, *r_pre_in;
  void *dx, *df, *dg, *dw_post, *dw_pre;
  float *part;   // workspace: [blocks][2][norm_part_row(d)] column sums of a block's rows (NULL: none wanted)
  float *terms;  // workspace: [rows][4] terms of long rows
};
// Floats of one row of column sums: 16-byte pieces, and room for rows that start
// inside one.
inline __host__ __device__ long norm_part_row(int d) { return (d + 15L) & ~7L; }
// Blocks that leave column sums: four per SM of the part, more where rows are short.
inline __host__ __device__ int norm_max_blocks(int d) { return 152 * (d >= 2048 ? 4 : (d >= 1024 ? 8 : 16)); }
// Columns from which the backward takes two launches.
inline __host__ __device__ int norm_long(int dtype) { return dtype == MOE_ELEM_FP32 ? 4096 : 8192; }
cudaError_t launch_norm_forward(const NormArgs &a, int num_sms, cudaStream_t s);
cudaError_t launch_norm_backward(const NormArgs &a, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------- embedding
struct EmbedArgs {
  int rows, V, d, dtype, grad_dtype, ids64, accumulate;
  float scale;
  long ld_t, ld_o;
  const void *ids, *table, *dout;
  void *out, *dtable;
  // workspace of the backward (offsets from embed_workspace)
  uint8_t *ws;
};
size_t embed_workspace(int rows, long V, int d);
cudaError_t launch_embed_forward(const EmbedArgs &a, cudaStream_t s);
cudaError_t launch_embed_backward(const EmbedArgs &a, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------- loss over a vocabulary
// The rows that count (a label inside the vocabulary; backward: a gradient too)
// stand first in a padded copy of x; everything after that works on the copy.
// `pad` is rows rounded up to 256; width a multiple of 256.
struct VocabArgs {
  int rows, V, d, dtype, grad_dtype, labels64, accumulate;
  long ld_x, ld_w, ld_dx;
  const void *x, *w, *labels;
  const float *dloss, *dlse, *lse_in;
  float *loss, *lse;
  void *dx, *dw;
  // workspace
  int *status, *count;   // rows that count
  float *scale;          // what the backward's products are multiplied by in the end
  int *row, *place;      // [pad] row of a place, [rows] place of a row (-1: none)
  int *label;            // [pad]
  float *hit;            // [pad] the label's logit; backward: its dz
  float2 *part;          // forward: [rows][parts] (maximum, sum of exponentials) of 128 logits
  int parts;
  float *coef_p, *coef_l, *base;  // backward: [pad] dz = coef_p 2^(z log2 e - base), less coef_l for the label
  void *xs;              // [rows rounded up to 128][ld_xs] the copy of x
  void *ws_w;            // the padded copy of w where TMA cannot address it (else unused)
  void *dz;              // backward: [rows rounded up to 128][width] one piece of the logits' gradient
  float *sum;            // backward: [splits][rows][ld_sum] sums of dx
  long ld_xs, ld_ws_w, ld_sum;
  int width, splits;
  bool pad_w, vec_dw;
  // the piece at hand
  int v0, wp;
};
cudaError_t launch_vocab_forward(const VocabArgs &a, int num_sms, cudaStream_t s);
cudaError_t launch_vocab_backward(const VocabArgs &a, int num_sms, cudaStream_t s);
// The tensor-core products (vocab_tc.cu).
enum VocabMode { VOCAB_LOSS = 0, VOCAB_DZ = 1, VOCAB_DX = 2, VOCAB_DW = 3 };
cudaError_t launch_vocab_tc(const VocabArgs &a, int mode, cudaStream_t s);

// ---------------------------------------------------------------- norm of gradients, clipping
// Host arrays: addresses, lengths and types of the tensors; outs with out_dtypes
// (the tensor's type or fp32) for clipping.
struct GradTensors {
  int n;
  const void *const *data;
  void *const *outs;
  const int64_t *counts;
  const int32_t *dtypes, *out_dtypes;
};
size_t grad_workspace(int n);
cudaError_t launch_grads(const GradTensors &g, bool clip, double max_norm, double eps, float *norm, void *ws, int num_sms,
                         cudaStream_t s);

}  // namespace moe
