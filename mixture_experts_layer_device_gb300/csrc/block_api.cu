// Host side of the entry points around the layer (include/moe.h: moe_grouped_*,
// moe_norm_*, moe_embed_*): argument checks, workspace layouts and the choice
// of kernel.  Nothing here allocates memory or synchronises.
#include <math.h>

#include "block.h"
#include "elem.cuh"
#include "kernels.h"

namespace {

bool aligned(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }
constexpr int64_t kMaxStride = (1LL << 31) - 1;

// A row stride: 0 means contiguous.  False when it is not one.
bool stride(int64_t given, int64_t least, long *out) {
  *out = static_cast<long>(given == 0 ? least : given);
  return given == 0 || (given >= least && given <= kMaxStride);
}

// ---------------------------------------------------------------- grouped
struct GroupedWs {
  size_t status, tiles, order, maps, bytes;
};
GroupedWs grouped_ws(int E) {
  GroupedWs w;
  w.status = 0;
  w.tiles = 256;
  w.order = w.tiles + round256((3 * static_cast<size_t>(E) + 3) * 4);
  w.maps = w.order + round256(static_cast<size_t>(E) * 4);
  w.bytes = w.maps + static_cast<size_t>(E) * 2 * 128 + 128;  // aligned to 128 bytes in place
  return w;
}

int grouped_check(const moe_grouped_config *c, moe::GroupedArgs *g) {
  if (!c) return MOE_ERR_ARG;
  if (c->rows < 0 || c->E <= 0 || c->N <= 0 || c->K <= 0) return MOE_ERR_ARG;
  if (c->dtype != MOE_ELEM_BF16 && c->dtype != MOE_ELEM_FP16) return MOE_ERR_ARG;
  if (c->out_dtype != c->dtype && c->out_dtype != MOE_ELEM_FP32) return MOE_ERR_ARG;
  if (c->accumulate != 0 && (c->accumulate != 1 || c->out_dtype != MOE_ELEM_FP32)) return MOE_ERR_ARG;
  if (c->E > 32767 || c->N > (1 << 20) || c->K > (1 << 20) || c->rows >= (1LL << 31) - 256) return MOE_ERR_SHAPE;
  *g = moe::GroupedArgs();
  if (!stride(c->ld_x, c->K, &g->ld_x) || !stride(c->ld_y, c->N, &g->ld_y) || !stride(c->ld_w, c->K, &g->ld_w))
    return MOE_ERR_SHAPE;
  // tiles of the weight gradient are counted in 32 bits
  if (static_cast<int64_t>(c->E) * ((c->N + 255) / 256) * ((c->K + 255) / 256) >= (1LL << 30)) return MOE_ERR_SHAPE;
  // a matrix's extent may pass 2^31: only the strides of rows are held below it
  const int64_t extent = static_cast<int64_t>(c->N - 1) * g->ld_w + c->K;
  if (c->ld_e != 0 && (c->ld_e < extent || c->ld_e > (1LL << 40))) return MOE_ERR_SHAPE;
  g->ld_e = static_cast<long>(c->ld_e == 0 ? static_cast<int64_t>(c->N) * g->ld_w : c->ld_e);
  g->E = c->E;
  g->N = c->N;
  g->K = c->K;
  g->rows = static_cast<int>(c->rows);
  g->dtype = c->dtype;
  g->out_dtype = c->out_dtype;
  g->accumulate = c->accumulate;
  return MOE_OK;
}

void grouped_bind(moe::GroupedArgs *g, const int32_t *offsets, void *ws) {
  const GroupedWs w = grouped_ws(g->E);
  uint8_t *b = static_cast<uint8_t *>(ws);
  g->offsets = offsets;
  g->status = reinterpret_cast<int *>(b + w.status);
  g->tiles = reinterpret_cast<int *>(b + w.tiles);
  g->order = reinterpret_cast<int *>(b + w.order);
  g->maps = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(b + w.maps) + 127) & ~static_cast<uintptr_t>(127));
}

// TMA addresses rows of whole 16-byte units; the sizes that the products share
// decide for all of them, the pointers for each.
bool tma_rows(const void *p, long ld) { return aligned(p, 16) && ld % 8 == 0; }

bool grouped_tensor(const moe::GroupedArgs &g, int dir) {
  if (g.rows == 0 || g.N % 8 || g.K % 8) return false;
  const long widest = ((g.N > g.K ? g.N : g.K) + 255L) / 256;
  if ((g.rows / 256 + 2L * g.E) * widest >= (1L << 30)) return false;  // tiles are counted in 32 bits
  const bool w = tma_rows(g.w, g.ld_w) && g.ld_e % 8 == 0;
  if (dir == moe::GROUPED_FWD) return w && tma_rows(g.x, g.ld_x) && tma_rows(g.y, g.ld_y);
  if (dir == moe::GROUPED_DGRAD) return w && tma_rows(g.dy, g.ld_y) && tma_rows(g.dx, g.ld_x);
  return tma_rows(g.dy, g.ld_y) && tma_rows(g.x, g.ld_x) && aligned(g.dw, 16);
}

// Few rows that mostly have an expert of their own: reading the weights bounds
// the call and the tensor cores have nothing to reuse.
bool grouped_few(const moe::GroupedArgs &g) {
  return g.rows > 0 && g.rows <= 64 && g.rows <= 2L * g.E && g.K % 8 == 0 && tma_rows(g.x, g.ld_x) &&
         tma_rows(g.w, g.ld_w) && g.ld_e % 8 == 0;
}

int grouped_product(const moe::GroupedArgs &g, int dir, bool first, cudaStream_t s) {
  return status_of(grouped_tensor(g, dir) ? moe::launch_grouped_tc(g, dir, s)
                                          : moe::launch_grouped_plain(g, dir, first, s));
}

// ---------------------------------------------------------------- norm
int norm_check(const moe_norm_config *c, moe::NormArgs *a) {
  if (!c) return MOE_ERR_ARG;
  if (c->rows < 0 || c->d <= 0) return MOE_ERR_ARG;
  if (c->dtype < MOE_ELEM_BF16 || c->dtype > MOE_ELEM_FP32) return MOE_ERR_ARG;
  if (c->flags & ~(MOE_NORM_POST | MOE_NORM_PRE)) return MOE_ERR_ARG;
  if (c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_FULL) return MOE_ERR_ARG;
  if (!isfinite(c->alpha) || !(c->eps >= 0.f) || !isfinite(c->eps)) return MOE_ERR_ARG;
  if (c->d > 65536 || c->rows >= (1LL << 31)) return MOE_ERR_SHAPE;
  *a = moe::NormArgs();
  if (!stride(c->ld_x, c->d, &a->ld_x) || !stride(c->ld_f, c->d, &a->ld_f) || !stride(c->ld_z, c->d, &a->ld_z) ||
      !stride(c->ld_h, c->d, &a->ld_h) || !stride(c->ld_g, c->d, &a->ld_g))
    return MOE_ERR_SHAPE;
  a->rows = static_cast<int>(c->rows);
  a->d = c->d;
  a->dtype = c->dtype;
  a->flags = c->flags;
  a->gate = c->gate;
  a->alpha = c->alpha;
  a->eps = c->eps;
  return MOE_OK;
}

// ---------------------------------------------------------------- embedding
int embed_check(const moe_embed_config *c, moe::EmbedArgs *a) {
  if (!c) return MOE_ERR_ARG;
  if (c->rows < 0 || c->V <= 0 || c->d <= 0) return MOE_ERR_ARG;
  if (c->dtype < MOE_ELEM_BF16 || c->dtype > MOE_ELEM_FP32) return MOE_ERR_ARG;
  if (c->grad_dtype != c->dtype && c->grad_dtype != MOE_ELEM_FP32) return MOE_ERR_ARG;
  if ((c->ids64 != 0 && c->ids64 != 1) || (c->accumulate != 0 && c->accumulate != 1) || !isfinite(c->scale))
    return MOE_ERR_ARG;
  if (c->rows >= (1LL << 30) || c->V >= (1LL << 31) - 1 || c->d > (1 << 20)) return MOE_ERR_SHAPE;
  *a = moe::EmbedArgs();
  if (!stride(c->ld_t, c->d, &a->ld_t) || !stride(c->ld_o, c->d, &a->ld_o)) return MOE_ERR_SHAPE;
  a->rows = static_cast<int>(c->rows);
  a->V = static_cast<int>(c->V);
  a->d = c->d;
  a->dtype = c->dtype;
  a->grad_dtype = c->grad_dtype;
  a->ids64 = c->ids64;
  a->accumulate = c->accumulate;
  a->scale = c->scale;
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_grouped_workspace_bytes(const moe_grouped_config *cfg) {
  moe::GroupedArgs g;
  return grouped_check(cfg, &g) == MOE_OK ? grouped_ws(g.E).bytes : 0;
}

int moe_grouped_forward(const moe_grouped_config *cfg, const void *x, const void *w, const int32_t *offsets, void *y,
                        void *ws, moe_stream_t stream) {
  moe::GroupedArgs g;
  int rc = grouped_check(cfg, &g);
  if (rc != MOE_OK) return rc;
  if (g.accumulate) return MOE_ERR_ARG;  // a forward overwrites
  if (!w || !offsets || !ws || (g.rows && (!x || !y))) return MOE_ERR_ARG;
  if (!aligned(x, 2) || !aligned(w, 2) || !aligned(y, moe::elem_bytes(g.out_dtype)) || !aligned(offsets, 4) ||
      !aligned(ws, 16))
    return MOE_ERR_ALIGN;
  int sms;
  if ((rc = moe::host_device(&sms)) != MOE_OK) return rc;
  grouped_bind(&g, offsets, ws);
  g.x = x;
  g.w = w;
  g.y = y;
  if (grouped_few(g)) return status_of(moe::launch_grouped_few(g, stream));
  return grouped_product(g, moe::GROUPED_FWD, true, stream);
}

int moe_grouped_backward(const moe_grouped_config *cfg, const void *dy, const void *x, const void *w,
                         const int32_t *offsets, void *dx, void *dw, void *ws, moe_stream_t stream) {
  moe::GroupedArgs g;
  int rc = grouped_check(cfg, &g);
  if (rc != MOE_OK) return rc;
  if (!offsets || !ws || (g.rows && !dy)) return MOE_ERR_ARG;
  if (g.rows && !dx && !dw) return MOE_ERR_ARG;
  if ((dx && !w) || (dw && g.rows && !x)) return MOE_ERR_ARG;
  if (!aligned(dy, 2) || !aligned(x, 2) || !aligned(w, 2) || !aligned(dx, 2) ||
      !aligned(dw, moe::elem_bytes(g.out_dtype)) || !aligned(offsets, 4) || !aligned(ws, 16))
    return MOE_ERR_ALIGN;
  int sms;
  if ((rc = moe::host_device(&sms)) != MOE_OK) return rc;
  grouped_bind(&g, offsets, ws);
  g.dy = dy;
  g.x = x;
  g.w = w;
  g.dx = dx;
  g.dw = dw;
  if (dx && (rc = grouped_product(g, moe::GROUPED_DGRAD, true, stream)) != MOE_OK) return rc;
  if (dw && (rc = grouped_product(g, moe::GROUPED_WGRAD, !dx, stream)) != MOE_OK) return rc;
  return MOE_OK;
}

int moe_norm_forward(const moe_norm_config *cfg, const void *x, const void *f, const void *gate, const void *w_post,
                     const void *w_pre, void *z, void *h, float *r_post, float *r_pre, moe_stream_t stream) {
  moe::NormArgs a;
  int rc = norm_check(cfg, &a);
  if (rc != MOE_OK) return rc;
  const bool post = (a.flags & MOE_NORM_POST) != 0, pre = (a.flags & MOE_NORM_PRE) != 0;
  if (a.rows && (!x || (pre ? !h : !z))) return MOE_ERR_ARG;
  if (a.rows && ((post && !f) || (a.gate != MOE_GATE_NONE && (!f || !gate)))) return MOE_ERR_ARG;
  const int e = moe::elem_bytes(a.dtype);
  const void *elems[] = {x, f, gate, w_post, w_pre, z, h};
  for (const void *p : elems)
    if (!aligned(p, e)) return MOE_ERR_ALIGN;
  if (!aligned(r_post, 4) || !aligned(r_pre, 4)) return MOE_ERR_ALIGN;
  int sms;
  if ((rc = moe::host_device(&sms)) != MOE_OK) return rc;
  a.x = x;
  a.f = f;
  a.g = a.gate == MOE_GATE_NONE ? nullptr : gate;
  a.w_post = post ? w_post : nullptr;
  a.w_pre = pre ? w_pre : nullptr;
  a.z = z;
  a.h = pre ? h : nullptr;
  a.r_post = r_post;
  a.r_pre = r_pre;
  return status_of(moe::launch_norm_forward(a, sms, stream));
}

size_t moe_norm_workspace_bytes(const moe_norm_config *cfg) {
  moe::NormArgs a;
  if (norm_check(cfg, &a) != MOE_OK) return 0;
  const size_t slots = a.rows < moe::kNormMaxBlocks ? (a.rows > 0 ? a.rows + 3 : 1) : moe::kNormMaxBlocks;
  return slots * 2 * a.d * 4;
}

int moe_norm_backward(const moe_norm_config *cfg, const void *dz, const void *dh, const void *z, const void *f,
                      const void *gate, const void *w_post, const void *w_pre, const float *r_post,
                      const float *r_pre, void *dx, void *df, void *dgate, void *dw_post, void *dw_pre, void *ws,
                      moe_stream_t stream) {
  moe::NormArgs a;
  int rc = norm_check(cfg, &a);
  if (rc != MOE_OK) return rc;
  const bool post = (a.flags & MOE_NORM_POST) != 0, pre = (a.flags & MOE_NORM_PRE) != 0;
  if ((dw_post && !post) || (dw_pre && !pre) || (dgate && a.gate == MOE_GATE_NONE)) return MOE_ERR_ARG;
  const bool needs_f = df || dgate || dw_post;
  if (a.rows) {
    if (pre ? (!dh || !z || !r_pre) : !dz) return MOE_ERR_ARG;
    if (needs_f && (!f || (post && !r_post) || (a.gate != MOE_GATE_NONE && !gate))) return MOE_ERR_ARG;
  }
  const bool columns = dw_post || dw_pre || (dgate && a.gate == MOE_GATE_CHANNEL);
  if (columns && !ws) return MOE_ERR_ARG;
  if (columns && needs_f && a.gate == MOE_GATE_CHANNEL && !gate) return MOE_ERR_ARG;
  const int e = moe::elem_bytes(a.dtype);
  const void *elems[] = {dz, dh, z, f, gate, w_post, w_pre, dx, df, dgate, dw_post, dw_pre};
  for (const void *p : elems)
    if (!aligned(p, e)) return MOE_ERR_ALIGN;
  if (!aligned(r_post, 4) || !aligned(r_pre, 4) || !aligned(ws, 16)) return MOE_ERR_ALIGN;
  int sms;
  if ((rc = moe::host_device(&sms)) != MOE_OK) return rc;
  a.dz = dz;
  a.dh = pre ? dh : nullptr;
  a.zin = pre ? z : nullptr;
  a.f = needs_f ? f : nullptr;
  a.g = needs_f ? gate : nullptr;
  if (!needs_f || a.gate == MOE_GATE_NONE) {
    a.g = nullptr;
    a.gate = MOE_GATE_NONE;
  }
  if (!needs_f) a.flags &= ~MOE_NORM_POST;
  a.w_post = post && needs_f ? w_post : nullptr;
  a.w_pre = pre ? w_pre : nullptr;
  a.r_post_in = r_post;
  a.r_pre_in = r_pre;
  a.dx = dx;
  a.df = df;
  a.dg = dgate;
  a.dw_post = dw_post;
  a.dw_pre = dw_pre;
  a.part = columns ? static_cast<float *>(ws) : nullptr;
  return status_of(moe::launch_norm_backward(a, sms, stream));
}

int moe_embed_forward(const moe_embed_config *cfg, const void *ids, const void *table, void *out,
                      moe_stream_t stream) {
  moe::EmbedArgs a;
  int rc = embed_check(cfg, &a);
  if (rc != MOE_OK) return rc;
  if (!table || (a.rows && (!ids || !out))) return MOE_ERR_ARG;
  const int e = moe::elem_bytes(a.dtype);
  if (!aligned(ids, a.ids64 ? 8 : 4) || !aligned(table, e) || !aligned(out, e)) return MOE_ERR_ALIGN;
  int sms;
  if ((rc = moe::host_device(&sms)) != MOE_OK) return rc;
  a.ids = ids;
  a.table = table;
  a.out = out;
  return status_of(moe::launch_embed_forward(a, stream));
}

size_t moe_embed_workspace_bytes(const moe_embed_config *cfg) {
  moe::EmbedArgs a;
  return embed_check(cfg, &a) == MOE_OK ? moe::embed_workspace(a.rows, a.V, a.d) : 0;
}

int moe_embed_backward(const moe_embed_config *cfg, const void *ids, const void *dout, void *dtable, void *ws,
                       moe_stream_t stream) {
  moe::EmbedArgs a;
  int rc = embed_check(cfg, &a);
  if (rc != MOE_OK) return rc;
  if (!dtable || !ws || (a.rows && (!ids || !dout))) return MOE_ERR_ARG;
  if (!aligned(ids, a.ids64 ? 8 : 4) || !aligned(dout, moe::elem_bytes(a.dtype)) ||
      !aligned(dtable, moe::elem_bytes(a.grad_dtype)) || !aligned(ws, 16))
    return MOE_ERR_ALIGN;
  int sms;
  if ((rc = moe::host_device(&sms)) != MOE_OK) return rc;
  a.ids = ids;
  a.dout = dout;
  a.dtable = dtable;
  a.ws = static_cast<uint8_t *>(ws);
  return status_of(moe::launch_embed_backward(a, sms, stream));
}

}  // extern "C"
