// Host side of the entry points that end a training step (include/moe.h: moe_vocab_*,
// moe_grad_*): argument checks, workspace layouts, sizes of pieces.  Nothing
// here allocates device memory or synchronises.
#include <math.h>

#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include "block.h"
#include "elem.cuh"
#include "host_check.h"
#include "kernels.h"

namespace {

using moe::aligned;
using moe::round256;
using moe::status_of;
using moe::stride;

// ---------------------------------------------------------------- loss over a vocabulary
long pad8(long n) { return (n + 7) / 8 * 8; }
long tiles(long n) { return (n + 255) / 256; }

int vocab_check(const moe_vocab_config *c, moe::VocabArgs *a) {
  if (!c) return MOE_ERR_ARG;
  if (c->rows < 0 || c->V <= 0 || c->d <= 0) return MOE_ERR_ARG;
  if (c->dtype != MOE_ELEM_BF16 && c->dtype != MOE_ELEM_FP16) return MOE_ERR_ARG;
  if (c->grad_dtype != c->dtype && c->grad_dtype != MOE_ELEM_FP32) return MOE_ERR_ARG;
  if (c->accumulate != 0 && (c->accumulate != 1 || c->grad_dtype != MOE_ELEM_FP32)) return MOE_ERR_ARG;
  if ((c->labels64 != 0 && c->labels64 != 1) || (c->copy_w != 0 && c->copy_w != 1)) return MOE_ERR_ARG;
  if (c->rows >= (1LL << 30) || c->V >= (1LL << 30) || c->d > (1 << 20)) return MOE_ERR_SHAPE;
  // tiles are counted in 32 bits
  if (tiles(c->rows) * tiles(c->V) >= (1LL << 30) || tiles(c->rows) * tiles(c->d) >= (1LL << 30) ||
      tiles(c->V) * tiles(c->d) >= (1LL << 30))
    return MOE_ERR_SHAPE;
  *a = moe::VocabArgs();
  if (!stride(c->ld_x, c->d, &a->ld_x) || !stride(c->ld_w, c->d, &a->ld_w) || !stride(c->ld_dx, c->d, &a->ld_dx))
    return MOE_ERR_SHAPE;
  a->rows = static_cast<int>(c->rows);
  a->V = static_cast<int>(c->V);
  a->d = c->d;
  a->dtype = c->dtype;
  a->grad_dtype = c->grad_dtype;
  a->labels64 = c->labels64;
  a->accumulate = c->accumulate;
  a->pad_w = c->copy_w != 0;
  a->ld_xs = a->ld_ws_w = a->ld_sum = pad8(c->d);
  a->parts = static_cast<int>(2 * tiles(c->V));
  return MOE_OK;
}

// A piece of the vocabulary: as many entries as the gradient of the logits of all rows
// takes 512 MB for, 4096 at least (8192 rows, 5735 that count, 131072 x 4096: 11.41 ms with
// 128 MB, 11.25 with 256, 11.06 with 512, 10.97 with 1024, 11.07 with 2048).
constexpr int64_t kPieceBytes = 512LL << 20;
// DX: the piece's reduction is split so that the last round of tiles over the SM pairs is
// full; a split costs a pass of its sums through memory, taken as 2 %.
constexpr int kPairs = 76;
int vocab_splits(int64_t units, int64_t most) {
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= most && s <= 64; ++s) {
    const double rounds = static_cast<double>((units * s + kPairs - 1) / kPairs) / s * (1.0 + 0.02 * (s - 1));
    if (rounds < least) {
      least = rounds;
      best = s;
    }
    if (units * s >= 4 * kPairs) break;
  }
  return best;
}
void vocab_pieces(moe::VocabArgs *a) {
  const int64_t all = tiles(a->V) * 256;
  int64_t w = kPieceBytes / 2 / (a->rows > 0 ? a->rows : 1) / 256 * 256;
  if (w < 4096) w = 4096;
  a->width = static_cast<int>(w < all ? w : all);
  const int64_t units = tiles(a->rows > 0 ? a->rows : 1) * tiles(a->d);
  a->splits = vocab_splits(units, std::max<int64_t>(1, a->width / 512));
}

// Carves the workspace; returns its bytes.
size_t vocab_bind(moe::VocabArgs *a, bool backward, void *ws) {
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ws) + 255) & ~static_cast<uintptr_t>(255));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t *p = base + at;
    at += round256(bytes);
    return p;
  };
  const size_t rows = a->rows, pad = tiles(a->rows) * 256, high = (rows + 127) / 128 * 128;
  uint8_t *head = take(256);
  a->status = reinterpret_cast<int *>(head);
  a->count = reinterpret_cast<int *>(head + 4);
  a->scale = reinterpret_cast<float *>(head + 8);
  a->row = reinterpret_cast<int *>(take(pad * 4));
  a->label = reinterpret_cast<int *>(take(pad * 4));
  a->hit = reinterpret_cast<float *>(take(pad * 4));
  a->xs = take(high * a->ld_xs * 2);
  if (a->pad_w) a->ws_w = take(static_cast<size_t>(a->V) * a->ld_ws_w * 2);
  if (backward) {
    vocab_pieces(a);
    a->place = reinterpret_cast<int *>(take(rows * 4));
    a->coef_p = reinterpret_cast<float *>(take(pad * 4));
    a->coef_l = reinterpret_cast<float *>(take(pad * 4));
    a->base = reinterpret_cast<float *>(take(pad * 4));
    a->dz = take(high * a->width * 2);
    a->sum = reinterpret_cast<float *>(take(a->splits * rows * a->ld_sum * 4));
  } else {
    a->part = reinterpret_cast<float2 *>(take(rows * a->parts * 8));
  }
  return at + 256;
}

// The status word is the workspace's first: the carving starts there when ws is
// aligned to 256 bytes, which the entry points ask for.
int vocab_pointers(const moe::VocabArgs &a, const void *x, const void *w, const void *labels, const void *ws) {
  if (!w || !ws || (a.rows && (!x || !labels))) return MOE_ERR_ARG;
  if (!aligned(x, 2) || !aligned(w, 2) || !aligned(labels, a.labels64 ? 8 : 4) || !aligned(ws, 256)) return MOE_ERR_ALIGN;
  if (!a.pad_w && (!aligned(w, 16) || a.ld_w % 8 != 0)) return MOE_ERR_ALIGN;
  return MOE_OK;
}

// ---------------------------------------------------------------- gradients
int grad_check(const void *const *data, void *const *outs, const int64_t *counts, const int32_t *dtypes,
               const int32_t *out_dtypes, int32_t n, bool clip) {
  if (n < 0 || (n > 0 && (!data || !counts || !dtypes || (clip && (!outs || !out_dtypes))))) return MOE_ERR_ARG;
  if (n > (1 << 24)) return MOE_ERR_SHAPE;
  int64_t bytes = 0;
  for (int i = 0; i < n; ++i) {
    if (counts[i] < 0 || dtypes[i] < MOE_ELEM_BF16 || dtypes[i] > MOE_ELEM_FP32) return MOE_ERR_ARG;
    if (clip && out_dtypes[i] != dtypes[i] && out_dtypes[i] != MOE_ELEM_FP32) return MOE_ERR_ARG;
    if (counts[i] > (1LL << 42)) return MOE_ERR_SHAPE;
    if (counts[i] == 0) continue;
    if (!data[i] || (clip && !outs[i])) return MOE_ERR_ARG;
    if (!aligned(data[i], moe::elem_bytes(dtypes[i])) || (clip && !aligned(outs[i], moe::elem_bytes(out_dtypes[i]))))
      return MOE_ERR_ALIGN;
    // a launch's pieces of 32 KB are counted in 32 bits: the same large tensor many times over
    bytes += counts[i] * moe::elem_bytes(dtypes[i]);
    if (bytes > (1LL << 45)) return MOE_ERR_SHAPE;
  }
  return MOE_OK;
}

// Clipping writes every output from its own tensor only: outputs share no memory with
// one another nor with another tensor, and with their own they are the same.
bool grad_apart(const moe::GradTensors &g) {
  struct Span {
    uintptr_t from, to;
    int tensor;
    bool out;
  };
  std::vector<Span> spans;
  spans.reserve(2 * static_cast<size_t>(g.n));
  for (int i = 0; i < g.n; ++i) {
    if (g.counts[i] == 0) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(g.data[i]), b = reinterpret_cast<uintptr_t>(g.outs[i]);
    const uintptr_t na = g.counts[i] * moe::elem_bytes(g.dtypes[i]), nb = g.counts[i] * moe::elem_bytes(g.out_dtypes[i]);
    if (a == b && g.dtypes[i] == g.out_dtypes[i]) {
      spans.push_back({a, a + na, i, true});
    } else {
      spans.push_back({a, a + na, i, false});
      spans.push_back({b, b + nb, i, true});
    }
  }
  std::sort(spans.begin(), spans.end(), [](const Span &p, const Span &q) { return p.from < q.from; });
  uintptr_t end = 0, out_end = 0;  // of all spans so far, of the outputs so far
  for (const Span &p : spans) {
    if (p.from < out_end || (p.out && p.from < end)) return false;
    end = std::max(end, p.to);
    if (p.out) out_end = std::max(out_end, p.to);
  }
  return true;
}

}  // namespace

extern "C" {

size_t moe_vocab_forward_workspace_bytes(const moe_vocab_config *cfg) {
  moe::VocabArgs a;
  return vocab_check(cfg, &a) == MOE_OK ? vocab_bind(&a, false, nullptr) : 0;
}

size_t moe_vocab_backward_workspace_bytes(const moe_vocab_config *cfg) {
  moe::VocabArgs a;
  return vocab_check(cfg, &a) == MOE_OK ? vocab_bind(&a, true, nullptr) : 0;
}

int moe_vocab_forward(const moe_vocab_config *cfg, const void *x, const void *w, const void *labels, float *loss,
                      float *lse, void *ws, moe_stream_t stream) {
  moe::VocabArgs a;
  int rc = vocab_check(cfg, &a);
  if (rc != MOE_OK) return rc;
  if (a.rows && (!loss || !lse)) return MOE_ERR_ARG;
  if ((rc = vocab_pointers(a, x, w, labels, ws)) != MOE_OK) return rc;
  if (!aligned(loss, 4) || !aligned(lse, 4)) return MOE_ERR_ALIGN;
  int sms;
  if ((rc = moe::host_device(&sms)) != MOE_OK) return rc;
  vocab_bind(&a, false, ws);
  a.x = x;
  a.w = w;
  a.labels = labels;
  a.loss = loss;
  a.lse = lse;
  a.v0 = 0;
  a.wp = a.V;
  return status_of(moe::launch_vocab_forward(a, sms, stream));
}

int moe_vocab_backward(const moe_vocab_config *cfg, const float *dloss, const float *dlse, const void *x, const void *w,
                       const void *labels, const float *lse, void *dx, void *dw, void *ws, moe_stream_t stream) {
  moe::VocabArgs a;
  int rc = vocab_check(cfg, &a);
  if (rc != MOE_OK) return rc;
  if (a.rows && ((!dloss && !dlse) || !lse)) return MOE_ERR_ARG;
  if (a.rows && !dx && !dw) return MOE_ERR_ARG;
  if ((rc = vocab_pointers(a, x, w, labels, ws)) != MOE_OK) return rc;
  if (!aligned(dloss, 4) || !aligned(dlse, 4) || !aligned(lse, 4) || !aligned(dx, 2) ||
      !aligned(dw, moe::elem_bytes(a.grad_dtype)))
    return MOE_ERR_ALIGN;
  int sms;
  if ((rc = moe::host_device(&sms)) != MOE_OK) return rc;
  vocab_bind(&a, true, ws);
  a.x = x;
  a.w = w;
  a.labels = labels;
  a.dloss = dloss;
  a.dlse = dlse;
  a.lse_in = lse;
  a.dx = dx;
  a.dw = dw;
  a.vec_dw = aligned(dw, 16) && a.d * moe::elem_bytes(a.grad_dtype) % 16 == 0;
  return status_of(moe::launch_vocab_backward(a, sms, stream));
}

size_t moe_grad_workspace_bytes(int32_t n) { return n < 0 || n > (1 << 24) ? 0 : moe::grad_workspace(n); }

int moe_grad_norm(const void *const *grads, const int64_t *counts, const int32_t *dtypes, int32_t n, float *norm,
                  void *ws, moe_stream_t stream) {
  int rc = grad_check(grads, nullptr, counts, dtypes, nullptr, n, false);
  if (rc != MOE_OK) return rc;
  if (!norm || !ws) return MOE_ERR_ARG;
  if (!aligned(norm, 4) || !aligned(ws, 16)) return MOE_ERR_ALIGN;
  int sms;
  if ((rc = moe::host_device(&sms)) != MOE_OK) return rc;
  const moe::GradTensors g = {n, grads, nullptr, counts, dtypes, nullptr};
  return status_of(moe::launch_grads(g, false, 0.0, 0.0, norm, ws, sms, stream));
}

int moe_grad_clip(const moe_clip_config *cfg, const void *const *grads, void *const *outs, const int64_t *counts,
                  const int32_t *dtypes, const int32_t *out_dtypes, int32_t n, float *norm, void *ws,
                  moe_stream_t stream) {
  if (!cfg) return MOE_ERR_ARG;
  int rc = grad_check(grads, outs, counts, dtypes, out_dtypes, n, true);
  if (rc != MOE_OK) return rc;
  if (!norm || !ws || !(cfg->max_norm >= 0.0) || !(cfg->eps > 0.0) || !isfinite(cfg->eps)) return MOE_ERR_ARG;
  if (!aligned(norm, 4) || !aligned(ws, 16)) return MOE_ERR_ALIGN;
  const moe::GradTensors g = {n, grads, outs, counts, dtypes, out_dtypes};
  try {
    if (!grad_apart(g)) return MOE_ERR_ARG;
  } catch (const std::bad_alloc &) {
    return MOE_ERR_ARG;
  }
  int sms;
  if ((rc = moe::host_device(&sms)) != MOE_OK) return rc;
  return status_of(moe::launch_grads(g, true, cfg->max_norm, cfg->eps, norm, ws, sms, stream));
}

}  // extern "C"
