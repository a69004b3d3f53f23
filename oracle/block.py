"""The operators around the layer in float64: ragged products grouped by
expert, the norms around a block with gate and residual scale, the token
embedding, each with its gradient.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The pages have no counterpart of these; the definitions are

* grouped: y[r] = x[r] W[e]^T for offsets[e] <= r < offsets[e + 1], 0 for a row
  of no expert; dx[r] = dy[r] W[e]; dW[e] = sum_r dy[r]^T x[r];
* norm: n = w_post f / rms(f), z = alpha x + g n, h = w_pre z / rms(z) with
  rms(v) = sqrt(mean(v^2) + eps), either norm left out on request;
* embedding: out[t] = scale table[ids[t]], 0 for an id outside the table.

The ``*_size`` results are the same expressions over absolute values: what a
rounding error of the fp32 sums is proportional to.
"""
import numpy as np


def grouped_forward(x, W, offsets):
    """(y, size of the sums)."""
    y = np.zeros((x.shape[0], W.shape[1]))
    size = np.zeros_like(y)
    for e in range(W.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        y[lo:hi] = x[lo:hi] @ W[e].T
        size[lo:hi] = np.abs(x[lo:hi]) @ np.abs(W[e]).T
    return y, size


def grouped_backward(dy, x, W, offsets):
    """(dx, dW, sizes of both)."""
    dx, dW = np.zeros((x.shape[0], W.shape[2])), np.zeros(W.shape)
    sx, sW = np.zeros_like(dx), np.zeros_like(dW)
    for e in range(W.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        dx[lo:hi] = dy[lo:hi] @ W[e]
        sx[lo:hi] = np.abs(dy[lo:hi]) @ np.abs(W[e])
        dW[e] = dy[lo:hi].T @ x[lo:hi]
        sW[e] = np.abs(dy[lo:hi]).T @ np.abs(x[lo:hi])
    return dx, dW, sx, sW


def _gate(gate, kind):
    if kind == "none":
        return np.ones(())
    return gate[:, None] if kind == "row" else gate


def norm_forward(x, f, gate, w_post, w_pre, kind="none", post=True, pre=True, alpha=1.0, eps=1e-6):
    """dict z, h, r_post, r_pre and the sizes z_size, h_size (None where absent)."""
    out = dict(h=None, r_post=None, r_pre=None, h_size=None)
    z, size = alpha * x, np.abs(alpha * x)
    if f is not None:
        n = f
        if post:
            out["r_post"] = 1.0 / np.sqrt((f * f).mean(1) + eps)
            n = f * out["r_post"][:, None] * (1.0 if w_post is None else w_post)
        gn = _gate(gate, kind) * n
        z, size = z + gn, size + np.abs(gn)
    out["z"], out["z_size"] = z, size
    if pre:
        out["r_pre"] = 1.0 / np.sqrt((z * z).mean(1) + eps)
        w = out["r_pre"][:, None] * (1.0 if w_pre is None else w_pre)
        out["h"], out["h_size"] = z * w, size * np.abs(w)
    return out


def norm_backward(dz, dh, z, f, gate, w_post, w_pre, r_post, r_pre, kind="none", post=True, pre=True, alpha=1.0):
    """dict dx, df, dgate, dw_post, dw_pre and their sizes (None where absent)."""
    like = dz if dz is not None else dh
    d = like.shape[1]
    wq = 1.0 if w_post is None else w_post
    wp = 1.0 if w_pre is None else w_pre
    t = np.zeros(like.shape) if dz is None else dz
    ts = np.abs(t)
    out = dict.fromkeys(["dx", "df", "dgate", "dw_post", "dw_pre"])
    size = dict.fromkeys(out)
    if pre:
        r = r_pre[:, None]
        u = wp * dh
        t = t + r * u - z * r ** 3 * (u * z).sum(1, keepdims=True) / d
        ts = ts + np.abs(r * u) + np.abs(z) * r ** 3 * np.abs(u * z).sum(1, keepdims=True) / d
        out["dw_pre"] = (dh * z * r).sum(0)
        size["dw_pre"] = np.abs(dh * z * r).sum(0)
    out["dx"], size["dx"] = alpha * t, np.abs(alpha) * ts
    if f is not None:
        r = r_post[:, None] if post else 1.0
        g = _gate(gate, kind)
        n = f * r * (wq if post else 1.0)
        a, s = t * n, ts * np.abs(n)
        if kind == "full":
            out["dgate"], size["dgate"] = a, s
        elif kind != "none":
            axis = 0 if kind == "channel" else 1
            out["dgate"], size["dgate"] = a.sum(axis), s.sum(axis)
        dn, dns = t * g, ts * np.abs(g)
        if post:
            out["dw_post"] = (dn * f * r).sum(0)
            size["dw_post"] = (dns * np.abs(f * r)).sum(0)
            u, us = wq * dn, np.abs(wq) * dns
            out["df"] = r * u - f * r ** 3 * (u * f).sum(1, keepdims=True) / d
            size["df"] = r * us + np.abs(f) * r ** 3 * (us * np.abs(f)).sum(1, keepdims=True) / d
        else:
            out["df"], size["df"] = dn, dns
    return out, size


def embed_forward(ids, table, scale=1.0):
    ids = np.asarray(ids).reshape(-1)
    ok = (ids >= 0) & (ids < table.shape[0])
    return np.where(ok[:, None], scale * table[np.where(ok, ids, 0)], 0.0)


def embed_backward(ids, dout, V, scale=1.0):
    """(dtable, size)."""
    ids = np.asarray(ids).reshape(-1)
    out, size = np.zeros((V, dout.shape[1])), np.zeros((V, dout.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < V:
            out[v] += scale * dout[t]
            size[v] += np.abs(scale * dout[t])
    return out, size
