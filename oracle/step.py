"""The operators that end a training step in float64, on torch tensors of any
device: the loss over a vocabulary, the gated products grouped by expert, the
norm of all gradients and their clipping.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

* vocab: z = x W^T, lse_t = log sum_v exp z_tv, loss_t = lse_t - z_t[y_t];
  dz_tv = (dloss_t + dlse_t) exp(z_tv - lse_t) - dloss_t [v = y_t], dx = dz W,
  dW = dz^T x; a row whose label lies outside the vocabulary gives zeros;
* gated: g = x W_g^T, u = x W_u^T, h = act(g) u; dg = dh u act'(g), du = dh act(g);
* grad: norm = sqrt(sum g^2), c = min(1, max_norm / (norm + eps)).

The ``size`` results are the same expressions over absolute values: what a
rounding error of the fp32 sums is proportional to.
"""
import math

import torch

F = torch.float64


def act(kind, g):
    """(act(g), act'(g))."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if kind == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        # (1 + tanh(v)) / 2 is the logistic function of 2 v, which does not cancel
        a, b = 2 * math.sqrt(2 / math.pi), 0.044715
        s = torch.sigmoid(a * (g + b * g ** 3))
        return g * s, s + g * s * (1 - s) * a * (1 + 3 * b * g * g)
    return torch.clamp(g, min=0.0), (g > 0).to(g.dtype)


def vocab_forward(x, w, labels):
    """dict loss, lse, keep, and z_size: the largest sum of absolute terms of a row's logits."""
    keep = (labels >= 0) & (labels < w.shape[0])
    xs, ws = x[keep].to(F), w.to(F)
    z = xs @ ws.T
    lse, loss = (torch.zeros(x.shape[0], dtype=F, device=x.device) for _ in range(2))
    lse[keep] = torch.logsumexp(z, 1)
    loss[keep] = lse[keep] - z.gather(1, labels[keep].long()[:, None])[:, 0]
    size = torch.zeros_like(lse)
    size[keep] = (xs.abs() @ ws.abs().T).max(1).values
    return dict(loss=loss, lse=lse, keep=keep, z_size=size)


def vocab_backward(dloss, dlse, x, w, labels, lse, rounding, n_z):
    """dict dx, dw, tol_dx, tol_dw: how far the two may be off before their own rounding,
    from dz rounded by `rounding` of its value, logits off by n_z 2^-22 of their terms'
    sizes, exponentials by 2^-20, and fp32 sums."""
    zero = torch.zeros(x.shape[0], dtype=F, device=x.device)
    a = zero if dloss is None else dloss.to(F)
    b = a + (zero if dlse is None else dlse.to(F))
    keep = (labels >= 0) & (labels < w.shape[0]) & ((a != 0) | (b != 0))
    xs, ws, a, b = x[keep].to(F), w.to(F), a[keep, None], b[keep, None]
    z = xs @ ws.T
    p = torch.exp(z - lse[keep].to(F)[:, None])
    dz = b * p
    at = labels[keep].long()[:, None]
    dz.scatter_add_(1, at, -a)
    off = b.abs() * p * (n_z * 2.0 ** -22 * (xs.abs() @ ws.abs().T) + 2.0 ** -20 + 2.0 ** -22 * z.abs()) * 1.01
    top = torch.cat([a.abs(), b.abs()]).max() if a.numel() else 0.0
    off += rounding * dz.abs() + 2.0 ** -36 * top
    n, V = xs.shape[0], ws.shape[0]
    dx, dw = torch.zeros(x.shape, dtype=F, device=x.device), dz.T @ xs
    tol_dx, tol_dw = torch.zeros_like(dx), off.T @ xs.abs() + (n + 32) * 2.0 ** -22 * (dz.abs().T @ xs.abs())
    dx[keep] = dz @ ws
    tol_dx[keep] = off @ ws.abs() + (V + 32) * 2.0 ** -22 * (dz.abs() @ ws.abs())
    return dict(dx=dx, dw=dw, tol_dx=tol_dx, tol_dw=tol_dw)


def gated_forward(x, w, offsets, kind):
    """dict h, gu and their sizes; offsets a list."""
    m = w.shape[1] // 2
    gu = torch.zeros((x.shape[0], 2 * m), dtype=F, device=x.device)
    size = torch.zeros_like(gu)
    for e in range(w.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        gu[lo:hi] = x[lo:hi].to(F) @ w[e].to(F).T
        size[lo:hi] = x[lo:hi].to(F).abs() @ w[e].to(F).abs().T
    value, _ = act(kind, gu[:, :m])
    return dict(h=value * gu[:, m:], gu=gu, gu_size=size, value=value)


def gated_backward(dh, x, w, offsets, gu, kind, rounding):
    """dict dx, dw, tol_dx, tol_dw, from [dg, du] off by `rounding` of its value and 2^-20
    of its terms."""
    m = w.shape[1] // 2
    dx, dw = torch.zeros(x.shape, dtype=F, device=x.device), torch.zeros(w.shape, dtype=F, device=x.device)
    tx, tw = torch.zeros_like(dx), torch.zeros_like(dw)
    for e in range(w.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        g, u, d = gu[lo:hi, :m].to(F), gu[lo:hi, m:].to(F), dh[lo:hi].to(F)
        value, slope = act(kind, g)
        dgu = torch.cat([d * u * slope, d * value], 1)
        # the slope is a sum of two terms, each at most 1 + |g|
        off = rounding * dgu.abs() + 2.0 ** -20 * torch.cat([(d * u).abs() * (1 + g.abs()), (d * value).abs()], 1) + 2.0 ** -25
        xe, we = x[lo:hi].to(F), w[e].to(F)
        dx[lo:hi], dw[e] = dgu @ we, dgu.T @ xe
        tx[lo:hi] = off @ we.abs() + (2 * m + 32) * 2.0 ** -22 * (dgu.abs() @ we.abs())
        tw[e] = off.T @ xe.abs() + (hi - lo + 32) * 2.0 ** -22 * (dgu.abs().T @ xe.abs())
    return dict(dx=dx, dw=dw, tol_dx=tx, tol_dw=tw)


def grad_norm(grads):
    return math.sqrt(sum(float(g.to(F).square().sum()) for g in grads))


def grad_factor(grads, max_norm, eps):
    return min(1.0, max_norm / (grad_norm(grads) + eps))
