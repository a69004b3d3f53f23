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
  g->in_x = g->ld_x;
  g->in_y = g->ld_y;
  g->rows = static_cast<int>(c->rows);
  g->dtype = c->dtype;
  g->out_dtype = c->out_dtype;
  g->accumulate = c->accumulate;
  return MOE_OK;
}

// Operands whose row strides TMA cannot address are first copied into padded rows
// in the workspace, where the product is large against the copies.  Measured in
// bf16 at experts of [1057, 2001], us with copies / on the plain kernel, by the
// multiply-adds per copied element that the rule asks for 64 of:
//   forward   8000 rows, 16 experts (339): 97 / 352     100 experts (74): 282 / 517
//             2000 rows, 40 experts (48): 122 / 157     8000, 150 experts (51): 400 / 418
//             8000 rows, 300 experts (26): 763 / 747
//   dgrad     8000 rows, 150 experts (52): 390 / 507    300 experts (26): 747 / 943
//   wgrad     (copies no weights, 692)  2000 rows, 40 experts: 158 / 337
// The host does not know which experts have rows, so all their weights count as
// copied, though those of experts without rows are not.
long pad8(long n) { return (n + 7) / 8 * 8; }
struct GroupedPads {
  bool w, x, dy;  // the operands of the product whose strides need it
  bool worth;
};
GroupedPads grouped_pads(const moe::GroupedArgs &g, int dir) {
  GroupedPads p;
  p.w = dir != moe::GROUPED_WGRAD && (g.ld_w % 8 != 0 || g.ld_e % 8 != 0);
  p.x = dir != moe::GROUPED_DGRAD && g.ld_x % 8 != 0;
  p.dy = dir != moe::GROUPED_FWD && g.ld_y % 8 != 0;
  const double work = static_cast<double>(g.rows) * g.N * g.K;
  const double copied = (p.w ? static_cast<double>(g.E) * g.N * g.K : 0.0) + (p.x ? static_cast<double>(g.rows) * g.K : 0.0) +
                        (p.dy ? static_cast<double>(g.rows) * g.N : 0.0);
  p.worth = work >= 64.0 * copied && work >= 67108864.0;
  return p;
}

struct GroupedWs {
  size_t status, tiles, order, maps, w, x, dy, bytes;
};
GroupedWs grouped_ws(const moe::GroupedArgs &g) {
  GroupedWs l;
  const size_t E = g.E;
  l.status = 0;
  l.tiles = 256;
  l.order = l.tiles + round256((3 * E + 3) * 4);
  l.maps = l.order + round256((E + 1) * 4);
  l.w = l.maps + E * 2 * 128 + 256;  // maps and copies are aligned in place
  bool w = false, x = false, dy = false;
  for (int dir : {moe::GROUPED_FWD, moe::GROUPED_DGRAD, moe::GROUPED_WGRAD}) {
    const GroupedPads p = grouped_pads(g, dir);
    w |= p.worth && p.w;
    x |= p.worth && p.x;
    dy |= p.worth && p.dy;
  }
  l.x = l.w + (w ? round256(E * g.N * pad8(g.K) * 2) : 0);
  l.dy = l.x + (x ? round256(static_cast<size_t>(g.rows) * pad8(g.K) * 2) : 0);
  l.bytes = l.dy + (dy ? round256(static_cast<size_t>(g.rows) * pad8(g.N) * 2) : 0) + 256;
  return l;
}

void grouped_bind(moe::GroupedArgs *g, const int32_t *offsets, void *ws) {
  const GroupedWs w = grouped_ws(*g);
  uint8_t *b = static_cast<uint8_t *>(ws);
  g->offsets = offsets;
  g->status = reinterpret_cast<int *>(b + w.status);
  g->tiles = reinterpret_cast<int *>(b + w.tiles);
  g->order = reinterpret_cast<int *>(b + w.order);
  g->maps = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(b + w.maps) + 127) & ~static_cast<uintptr_t>(127));
}

// TMA addresses rows that start on 16-byte units.
bool tma_rows(const void *p, long ld) { return aligned(p, 16) && ld % 8 == 0; }

// Brings the operands of one product into TMA's form: true when the tensor-core
// kernel can run on *t (copies launched where needed; `have_dy`: dy's has been made).
// The copies mend strides only: an operand whose rows are whole 16-byte pieces but
// start inside one (a view from a column on) goes to the plain kernel, whatever its size.
struct Padded {
  bool ok;
  int rc;
};
Padded grouped_tensor(const moe::GroupedArgs &g, int dir, uint8_t *ws, moe::GroupedArgs *t, bool *have_dy, cudaStream_t s) {
  *t = g;
  if (g.rows == 0) return {false, MOE_OK};
  const long widest = ((g.N > g.K ? g.N : g.K) + 255L) / 256;
  if ((g.rows / 256 + 2L * g.E) * widest >= (1L << 30)) return {false, MOE_OK};  // tiles are counted in 32 bits
  const bool uw = dir != moe::GROUPED_WGRAD, ux = dir != moe::GROUPED_DGRAD, uy = dir != moe::GROUPED_FWD;
  const GroupedPads p = grouped_pads(g, dir);
  if ((p.w || p.x || p.dy) && !p.worth) return {false, MOE_OK};
  if ((uw && !p.w && !aligned(g.w, 16)) || (ux && !p.x && !aligned(g.x, 16)) || (uy && !p.dy && !aligned(g.dy, 16)))
    return {false, MOE_OK};
  const GroupedWs l = grouped_ws(g);
  auto place = [&](size_t at) {
    return reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(ws) + at + 127) & ~static_cast<uintptr_t>(127));
  };
  cudaError_t e = cudaSuccess;
  if (p.w) {
    t->w = place(l.w);
    t->ld_w = pad8(g.K);
    t->ld_e = g.N * t->ld_w;
    e = moe::launch_grouped_pad(g, g.w, static_cast<long>(g.E) * g.N, g.K, g.ld_w, true, const_cast<void *>(t->w), t->ld_w, s);
  }
  // the strides of x and dx, y and dy are shared: an output keeps its own
  if (e == cudaSuccess && p.x) {
    t->x = place(l.x);
    t->in_x = pad8(g.K);
    e = moe::launch_grouped_pad(g, g.x, g.rows, g.K, g.ld_x, false, const_cast<void *>(t->x), t->in_x, s);
  }
  if (e == cudaSuccess && p.dy) {
    t->dy = place(l.dy);
    t->in_y = pad8(g.N);
    if (!*have_dy) e = moe::launch_grouped_pad(g, g.dy, g.rows, g.N, g.ld_y, false, const_cast<void *>(t->dy), t->in_y, s);
    *have_dy = true;
  }
  if (e != cudaSuccess) return {false, MOE_ERR_CUDA};
  if (dir == moe::GROUPED_FWD) t->vec_out = tma_rows(g.y, g.ld_y) && g.N % 8 == 0;
  else if (dir == moe::GROUPED_DGRAD) t->vec_out = tma_rows(g.dx, g.ld_x) && g.K % 8 == 0;
  else t->vec_out = aligned(g.dw, 16) && g.K % 8 == 0;
  return {true, MOE_OK};
}

// Few rows: reading the weights bounds the call, and the tensor cores have little to
// reuse.  By the average over all experts, as the offsets are on the device.  Measured at
// experts of [2048, 4096] in bf16, us here / on the tensor cores:
//                            rows spread over the experts   all on one expert
//   8 experts, 1 row         11 / 27
//   8 experts, 16 rows       28 / 32                        19 / 27
//   32 experts, 64 rows      84 / 102                       48 / 27
//   512 experts, 10 rows     30 / 54                        17 / 27
//   512 experts, 32 rows     82 / 103                       33 / 27
//   512 experts, 64 rows     152 / 178                      53 / 27
// An expert's weights are read again for every four of its rows: from some 25 rows of one
// expert on (a call whose rows all take one adapter) the tensor cores would be faster.
bool grouped_few(const moe::GroupedArgs &g) {
  return g.rows > 0 && g.rows <= 64 && g.rows <= 2L * g.E && g.K % 8 == 0 && tma_rows(g.x, g.ld_x) &&
         tma_rows(g.w, g.ld_w) && g.ld_e % 8 == 0;
}

// One product: t on the tensor cores when that can be, else g on the plain kernel.
int grouped_product(const Padded &p, const moe::GroupedArgs &t, const moe::GroupedArgs &g, int dir, bool first,
                    int sms, cudaStream_t s) {
  if (p.ok) return status_of(moe::launch_grouped_tc(t, dir, sms, s));
  if (dir == moe::GROUPED_WGRAD && g.zeroed) {
    int rc = status_of(moe::launch_grouped_order(g, s));
    if (rc == MOE_OK) rc = status_of(moe::launch_grouped_zero(g, sms, s));
    if (rc != MOE_OK) return rc;
  }
  return status_of(moe::launch_grouped_plain(g, dir, first, s));
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

size_t norm_part_bytes(const moe::NormArgs &a) {
  const int most = moe::norm_max_blocks(a.d);
  const size_t slots = a.rows < most ? (a.rows > 0 ? a.rows : 1) : most;
  return round256(slots * 2 * moe::norm_part_row(a.d) * 4);
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
  return grouped_check(cfg, &g) == MOE_OK ? grouped_ws(g).bytes : 0;
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
  bool have_dy = false;
  moe::GroupedArgs t;
  const Padded p = grouped_tensor(g, moe::GROUPED_FWD, static_cast<uint8_t *>(ws), &t, &have_dy, stream);
  return p.rc != MOE_OK ? p.rc : grouped_product(p, t, g, moe::GROUPED_FWD, true, sms, stream);
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
  // Large weight gradients: the experts without rows are written by plain stores (6.9
  // TB/s) and left out of the product, whose epilogue reaches 2.8 to 6.1 TB/s on zeros.
  g.zeroed = dw && !g.accumulate && static_cast<double>(g.E) * g.N * g.K >= 16e6;
  bool have_dy = false;
  moe::GroupedArgs dg, wg;
  Padded pd = {false, MOE_OK}, pw = {false, MOE_OK};
  if (dx) pd = grouped_tensor(g, moe::GROUPED_DGRAD, static_cast<uint8_t *>(ws), &dg, &have_dy, stream);
  if (pd.rc == MOE_OK && dw) pw = grouped_tensor(g, moe::GROUPED_WGRAD, static_cast<uint8_t *>(ws), &wg, &have_dy, stream);
  if (pd.rc != MOE_OK || pw.rc != MOE_OK) return pd.rc != MOE_OK ? pd.rc : pw.rc;
  if (pd.ok && pw.ok) return status_of(moe::launch_grouped_tc_pair(dg, wg, sms, stream));
  if (dx && (rc = grouped_product(pd, dg, g, moe::GROUPED_DGRAD, true, sms, stream)) != MOE_OK) return rc;
  if (dw && (rc = grouped_product(pw, wg, g, moe::GROUPED_WGRAD, !dx, sms, stream)) != MOE_OK) return rc;
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
  return norm_part_bytes(a) + (a.d > moe::norm_long(a.dtype) ? static_cast<size_t>(a.rows) * 16 : 0);
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
  if (!ws) return MOE_ERR_ARG;
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
  a.terms = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + norm_part_bytes(a));
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
