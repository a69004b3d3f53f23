"""What a model needs around the MoE layer, on torch tensors: ragged matrix
products grouped by expert, plain and gated, the norms around a block with its
gate and residual scale, the token embedding with its gradient, the loss over
the vocabulary with its gradients, and the norm and clipping of all gradients
(include/moe.h: moe_grouped_*, moe_gated_*, moe_norm_*, moe_embed_*,
moe_vocab_*, moe_grad_*).

Plain functions: they check their arguments, allocate outputs and workspaces
from torch and call the library; all arithmetic runs in its kernels.  They run
on torch's current stream and do not synchronise; with `stream` (a stream or its
handle) they run as under `torch.cuda.stream(stream)`: what they read has to be
ready on it, and what they return is.  All tensors of a call are on the current
GPU.  Where a call changes a tensor's values in place (clipping, accumulate=True) autograd
is told.  The autograd functions and modules over them are in module.py.
"""
import ctypes
from array import array
from functools import lru_cache
from operator import attrgetter

import torch

from . import (ACTS, GATES, MOE_ELEM_BF16, MOE_ELEM_FP16, MOE_ELEM_FP32, MOE_NORM_POST, MOE_NORM_PRE, MoeClipConfig,
               MoeEmbedConfig, MoeGatedConfig, MoeGroupedConfig, MoeNormConfig, MoeVocabConfig, _stream, check, lib, moe_get_status)

_ELEM = {torch.bfloat16: MOE_ELEM_BF16, torch.float16: MOE_ELEM_FP16, torch.float32: MOE_ELEM_FP32}


def _bad(what, *args):
    raise ValueError(what % args if args else what)


_current_gpu = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _gpu(t, name):
    """The index of the GPU of a call's first tensor: the current one, on which the library launches."""
    gpu = t.get_device()
    if gpu < 0 or gpu != _current_gpu():
        _bad("%s is on %s, not on the current GPU", name, t.device)
    return gpu


def _rows(t, name, cols, gpu, dtype=None, rows=None):
    """A 2-D matrix on the call's GPU whose rows are contiguous; its row stride."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or (rows is not None and shape[0] != rows):
        _bad("%s has shape %s, expected [%s, %d]", name, tuple(shape), "rows" if rows is None else rows, cols)
    if dtype is not None and t.dtype != dtype:
        _bad("%s is %s, expected %s", name, t.dtype, dtype)
    if t.get_device() != gpu:
        _bad("%s is on %s, expected GPU %d", name, t.device, gpu)
    if t.is_contiguous():
        return t, cols
    if (t.stride(1) != 1 and cols > 1) or (shape[0] > 1 and t.stride(0) < cols):
        return t.contiguous(), cols
    return t, (t.stride(0) if shape[0] > 1 else cols)


def _narrow(t, ld):
    """A matrix whose gradient is allocated with its row stride (the library has one for
    the two); its row stride.  Copied where that would be more than eight times the
    memory: parts of a fused buffer keep their stride, as a copy costs time (8192 x 4096:
    the grouped backward takes 329 us, 401 with it; 16384 x 6144: the norms' 177, 384)."""
    return (t.contiguous(), t.shape[1]) if ld > 8 * t.shape[1] else (t, ld)


def _out(t, name, rows, cols, dtype, device, gpu):
    """The caller's output matrix (rows contiguous), or a new one; its row stride."""
    if t is None:
        return torch.empty((rows, cols), dtype=dtype, device=device), cols
    if not (t.shape == (rows, cols) and t.dtype == dtype and t.get_device() == gpu and
            (cols == 1 or t.stride(1) == 1) and (rows <= 1 or t.stride(0) >= cols)):
        _bad("%s must be a %s matrix [%d, %d] with contiguous rows on GPU %d", name, dtype, rows, cols, gpu)
    return t, (t.stride(0) if rows > 1 else cols)


def _vector(t, name, n, dtype, gpu):
    if t is None:
        return None
    if t.shape != (n,) or t.dtype != dtype or t.get_device() != gpu:
        _bad("%s must be a %s vector of %d on GPU %d", name, dtype, n, gpu)
    return t.contiguous()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _plan(cfg, workspace_bytes):
    """(the config, a reference to it for the library's calls, the call's workspace
    bytes): what depends on sizes, types and strides alone, kept for the next call."""
    ref = ctypes.byref(cfg)
    return cfg, ref, workspace_bytes(ref) if workspace_bytes else 0


def _ws(plan, device):
    if plan[2] <= 0:
        _bad("the library does not take these sizes")
    return torch.empty(plan[2], dtype=torch.uint8, device=device)


# The library writes through addresses: autograd is told of the callers' tensors whose values
# a call changes in place, so that a graph which has saved one refuses its stale values.
_changed = torch.autograd.graph.increment_version


def _on(stream, call, *args, **kw):
    """The whole call with `stream` as the current one, so that the copies it makes,
    its outputs and its workspace are in order with its kernels.  The caller's
    tensors are kept until `stream` has used them, the results until the caller's
    current stream has."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    caller = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    for a in (*args, *kw.values()):
        for t in a if isinstance(a, (list, tuple)) else (a,):
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None:
            t.record_stream(caller)
    return out


# ---------------------------------------------------------------- grouped products
@lru_cache(maxsize=512)
def _grouped_plan(*fields):
    return _plan(MoeGroupedConfig(*fields), lib().moe_grouped_workspace_bytes)


def _grouped(x, w, offsets, name):
    x_dtype = x.dtype
    if not (x_dtype in (torch.bfloat16, torch.float16)):
        _bad("%s must be bfloat16 or float16", name)
    gpu = _gpu(x, name)
    if not (w.dim() == 3 and w.dtype == x_dtype and w.get_device() == gpu):
        _bad("w must be a %s tensor [E, N, K] on GPU %d", x_dtype, gpu)
    E, N, K = w.shape
    if not (offsets.dim() == 1 and offsets.shape[0] == E + 1 and offsets.dtype == torch.int32 and
            offsets.get_device() == gpu):
        _bad("offsets must be an int32 vector of E + 1 = %d on GPU %d", E + 1, gpu)
    if (K > 1 and w.stride(2) != 1) or (N > 1 and w.stride(1) < K) or \
            (E > 1 and w.stride(0) < (N - 1) * w.stride(1) + K):
        w = w.contiguous()
    return gpu, w, offsets.contiguous(), E, N, K, (w.stride(1) if N > 1 else K)


def grouped_forward(x, w, offsets, *, out=None, out_dtype=None, return_workspace=False, stream=None):
    """y [rows, N]: y[r] = x[r] w[e]^T for the rows offsets[e] <= r < offsets[e + 1]
    of expert e (0 for a row of no expert).  x [rows, K] and w [E, N, K] bf16 or
    fp16, offsets int32 [E + 1] on the GPU as moe_route writes them; y of x's
    type or fp32 (out_dtype, or out's).  Rows of w (and of x, from a column on) may
    be strided; a w whose last two dimensions lie in the other order is copied
    whole in every call."""
    if stream is not None:
        return _on(stream, grouped_forward, x, w, offsets, out=out, out_dtype=out_dtype, return_workspace=return_workspace)
    gpu, w, offsets, E, N, K, ld_w = _grouped(x, w, offsets, "x")
    x, ld_x = _rows(x, "x", K, gpu)
    out_dtype = out_dtype or (out.dtype if out is not None else x.dtype)
    if not (out_dtype in (x.dtype, torch.float32)):
        _bad("y is of x's type or float32")
    y, ld_y = _out(out, "out", x.shape[0], N, out_dtype, x.device, gpu)
    ld_e = w.stride(0) if E > 1 else 0
    plan = _grouped_plan(x.shape[0], E, N, K, _ELEM[x.dtype], _ELEM[out_dtype], 0, ld_x, ld_y, ld_w, ld_e)
    ws = _ws(plan, x.device)
    check(lib().moe_grouped_forward(plan[1], x.data_ptr(), w.data_ptr(), offsets.data_ptr(), y.data_ptr(),
                                    ws.data_ptr(), _stream(None)))
    return (y, ws) if return_workspace else y


def _product_grads(x, ld_x, rows, E, N, K, dtype, gpu, dx, dw, need_dx, need_dw, dw_dtype, accumulate, name):
    """(x, its row stride, dx, dw) of a backward: the outputs checked or allocated, None
    where not needed, x copied where dx cannot share its stride."""
    dw_dtype = dw_dtype or (dw.dtype if dw is not None else dtype)
    if not (dw_dtype in (dtype, torch.float32)):
        _bad("dw is of %s's type or float32", name)
    if not (not accumulate or (dw is not None and dw_dtype == torch.float32)):
        _bad("accumulate adds to a given float32 dw")
    if not (need_dx or need_dw):
        _bad("nothing to compute")
    if need_dx:
        if dx is None:
            x, ld_x = _narrow(x, ld_x)
            dx = torch.empty((rows, ld_x), dtype=dtype, device=x.device)
            dx = dx if ld_x == K else dx[:, :K]
        if not (dx.shape == (rows, K) and dx.dtype == dtype and dx.get_device() == gpu and
                (K == 1 or dx.stride(1) == 1)):
            _bad("dx must be a %s matrix [%d, %d] with contiguous rows on GPU %d", dtype, rows, K, gpu)
        if rows > 1 and dx.stride(0) != ld_x:
            x, ld_x = x.contiguous(), K
            if not (dx.stride(0) == K):
                _bad("dx must have x's row stride or be contiguous")
    if need_dw:
        if dw is None:
            dw = torch.empty((E, N, K), dtype=dw_dtype, device=x.device)
        if not (dw.shape == (E, N, K) and dw.dtype == dw_dtype and dw.get_device() == gpu and dw.is_contiguous()):
            _bad("dw must be a contiguous %s tensor [%d, %d, %d] on GPU %d", dw_dtype, E, N, K, gpu)
    return x, ld_x, dx if need_dx else None, dw if need_dw else None


def grouped_backward(dy, x, w, offsets, *, dx=None, dw=None, need_dx=True, need_dw=True, dw_dtype=None,
                     accumulate=False, return_workspace=False, stream=None):
    """(dx [rows, K], dw [E, N, K]) of grouped_forward: dx[r] = dy[r] w[e], dw[e] =
    sum of dy[r]^T x[r] over e's rows (zeros for an expert without rows), either
    None when not needed.  dw is of x's type or fp32 (dw_dtype, or dw's); with
    accumulate it must be given, fp32, and is added to."""
    if stream is not None:
        return _on(stream, grouped_backward, dy, x, w, offsets, dx=dx, dw=dw, need_dx=need_dx, need_dw=need_dw,
                   dw_dtype=dw_dtype, accumulate=accumulate, return_workspace=return_workspace)
    gpu, w, offsets, E, N, K, ld_w = _grouped(dy, w, offsets, "dy")
    rows = dy.shape[0]
    dy, ld_y = _rows(dy, "dy", N, gpu)
    x, ld_x = _rows(x, "x", K, gpu, dy.dtype, rows)
    x, ld_x, dx, dw = _product_grads(x, ld_x, rows, E, N, K, dy.dtype, gpu, dx, dw, need_dx, need_dw, dw_dtype, accumulate,
                                     "dy")
    ld_e = w.stride(0) if E > 1 else 0
    plan = _grouped_plan(rows, E, N, K, _ELEM[dy.dtype], _ELEM[dw.dtype if need_dw else dy.dtype], int(accumulate), ld_x,
                         ld_y, ld_w, ld_e)
    ws = _ws(plan, dy.device)
    check(lib().moe_grouped_backward(plan[1], dy.data_ptr(), x.data_ptr(), w.data_ptr(), offsets.data_ptr(), _ptr(dx),
                                     _ptr(dw), ws.data_ptr(), _stream(None)))
    if accumulate and need_dw:
        _changed(dw)
    return (dx, dw, ws) if return_workspace else (dx, dw)


def grouped_status(ws, stream=None):
    """Synchronises the current stream, or `stream`: the one that the call ran on.  The
    device status of the call that used workspace `ws` (return_workspace=True): 0, or
    -7 when its offsets descend or leave the rows."""
    return moe_get_status(ws, stream)


# ---------------------------------------------------------------- gated products
@lru_cache(maxsize=512)
def _gated_plan(backward, *fields):
    return _plan(MoeGatedConfig(*fields), lib().moe_gated_backward_workspace_bytes if backward
                 else lib().moe_gated_forward_workspace_bytes)


def _gated(x, w, offsets, act, name):
    gpu, w, offsets, E, N, K, ld_w = _grouped(x, w, offsets, name)
    if N % 2:
        _bad("w has %d rows per expert, expected the gate's and as many of the up projection", N)
    if not (act in ACTS):
        _bad("act is one of %s", sorted(ACTS))
    return gpu, w, offsets, E, N // 2, K, ld_w


def gated_forward(x, w, offsets, *, act="silu", need_gu=True, out=None, gu=None, return_workspace=False, stream=None):
    """(h [rows, m], gu [rows, 2m]): g = x[r] w[e][:m]^T, u = x[r] w[e][m:]^T, h = act(g) u
    for the rows offsets[e] <= r < offsets[e + 1] of expert e (0 for a row of no
    expert).  x [rows, K] and w [E, 2m, K] bf16 or fp16, offsets int32 [E + 1] as for
    grouped_forward; gu = [g, u] is what a backward needs (None without need_gu).
    act: "silu", "gelu", "gelu_tanh" or "relu"."""
    if stream is not None:
        return _on(stream, gated_forward, x, w, offsets, act=act, need_gu=need_gu, out=out, gu=gu,
                   return_workspace=return_workspace)
    gpu, w, offsets, E, m, K, ld_w = _gated(x, w, offsets, act, "x")
    x, ld_x = _rows(x, "x", K, gpu)
    rows, dt = x.shape[0], x.dtype
    h, ld_h = _out(out, "out", rows, m, dt, x.device, gpu)
    ld_gu = 2 * m
    if need_gu:
        gu, ld_gu = _out(gu, "gu", rows, 2 * m, dt, x.device, gpu)
    elif gu is not None:
        _bad("gu is given but not needed")
    el = _ELEM[dt]
    plan = _gated_plan(False, rows, E, m, K, el, el, ACTS[act], 0, ld_x, ld_h, ld_gu, ld_w, w.stride(0) if E > 1 else 0)
    ws = _ws(plan, x.device)
    check(lib().moe_gated_forward(plan[1], x.data_ptr(), w.data_ptr(), offsets.data_ptr(), h.data_ptr(), _ptr(gu),
                                  ws.data_ptr(), _stream(None)))
    return (h, gu, ws) if return_workspace else (h, gu)


def gated_backward(dh, x, w, offsets, gu, *, act="silu", dx=None, dw=None, need_dx=True, need_dw=True, dw_dtype=None,
                   accumulate=False, return_workspace=False, stream=None):
    """(dx [rows, K], dw [E, 2m, K]) of gated_forward from its gu, either None when not
    needed.  dw is of x's type or fp32 (dw_dtype, or dw's); with accumulate it must
    be given, fp32, and is added to."""
    if stream is not None:
        return _on(stream, gated_backward, dh, x, w, offsets, gu, act=act, dx=dx, dw=dw, need_dx=need_dx, need_dw=need_dw,
                   dw_dtype=dw_dtype, accumulate=accumulate, return_workspace=return_workspace)
    gpu, w, offsets, E, m, K, ld_w = _gated(dh, w, offsets, act, "dh")
    rows, dt = dh.shape[0], dh.dtype
    dh, ld_h = _rows(dh, "dh", m, gpu)
    x, ld_x = _rows(x, "x", K, gpu, dt, rows)
    gu, ld_gu = _rows(gu, "gu", 2 * m, gpu, dt, rows)
    x, ld_x, dx, dw = _product_grads(x, ld_x, rows, E, 2 * m, K, dt, gpu, dx, dw, need_dx, need_dw, dw_dtype, accumulate,
                                     "dh")
    plan = _gated_plan(True, rows, E, m, K, _ELEM[dt], _ELEM[dw.dtype if need_dw else dt], ACTS[act], int(accumulate),
                       ld_x, ld_h, ld_gu, ld_w, w.stride(0) if E > 1 else 0)
    ws = _ws(plan, dh.device)
    check(lib().moe_gated_backward(plan[1], dh.data_ptr(), x.data_ptr(), w.data_ptr(), offsets.data_ptr(), gu.data_ptr(),
                                   _ptr(dx), _ptr(dw), ws.data_ptr(), _stream(None)))
    if accumulate and need_dw:
        _changed(dw)
    return (dx, dw, ws) if return_workspace else (dx, dw)


# ---------------------------------------------------------------- block norms
@lru_cache(maxsize=512)
def _norm_plan(*fields):
    return _plan(MoeNormConfig(*fields), lib().moe_norm_workspace_bytes)


def _gate(gate, kind, rows, d, dtype, gpu):
    if not (kind in GATES):
        _bad("gate_kind is one of %s", sorted(GATES))
    if not ((gate is None) == (kind == "none")):
        _bad("a gate goes with its kind (channel, row or full)")
    if kind == "none":
        return None, d
    if kind == "full":
        return _rows(gate, "gate", d, gpu, dtype, rows)
    return _vector(gate, "gate", d if kind == "channel" else rows, dtype, gpu), d


def norm_forward(x, f=None, gate=None, w_post=None, w_pre=None, *, gate_kind="none", post=True, pre=True, alpha=1.0,
                 eps=1e-6, need_z=True, z=None, h=None, stream=None):
    """(z, h, r_post, r_pre):
        z = alpha x + g n,  n = w_post f / rms(f) (post) or f,  h = w_pre z / rms(z) (pre).
    x [rows, d] is the residual stream, f [rows, d] the block's output (None: z =
    alpha x), gate [d], [rows] or [rows, d] by gate_kind "channel", "row" or
    "full"; w_post and w_pre [d] or None (ones); all of one type (bf16, fp16,
    fp32).  r_post, r_pre [rows] fp32 are the reciprocal roots for the backward;
    what is not computed comes back as None."""
    if stream is not None:
        return _on(stream, norm_forward, x, f, gate, w_post, w_pre, gate_kind=gate_kind, post=post, pre=pre, alpha=alpha,
                   eps=eps, need_z=need_z, z=z, h=h)
    if not (x.dim() == 2 and x.dtype in _ELEM):
        _bad("x must be a bf16, fp16 or fp32 matrix [rows, d]")
    rows, d = x.shape
    gpu = _gpu(x, "x")
    x, ld_x = _rows(x, "x", d, gpu)
    ld_f, post = d, post and f is not None
    if f is not None:
        f, ld_f = _rows(f, "f", d, gpu, x.dtype, rows)
    if not (f is not None or gate is None):
        _bad("a gate needs the block's output f")
    if not (pre or need_z):
        _bad("nothing to compute")
    gate, ld_g = _gate(gate, gate_kind, rows, d, x.dtype, gpu)
    w_post = _vector(w_post, "w_post", d, x.dtype, gpu) if post else None
    w_pre = _vector(w_pre, "w_pre", d, x.dtype, gpu) if pre else None
    dev, ld_z, ld_h, r_post, r_pre = x.device, d, d, None, None
    if need_z:
        z, ld_z = _out(z, "z", rows, d, x.dtype, dev, gpu)
    if pre:
        h, ld_h = _out(h, "h", rows, d, x.dtype, dev, gpu)
        r_pre = torch.empty(rows, dtype=torch.float32, device=dev)
    if post:
        r_post = torch.empty(rows, dtype=torch.float32, device=dev)
    plan = _norm_plan(rows, d, _ELEM[x.dtype], (MOE_NORM_POST if post else 0) | (MOE_NORM_PRE if pre else 0),
                      GATES[gate_kind], float(alpha), float(eps), ld_x, ld_f, ld_z, ld_h, ld_g)
    z, h = z if need_z else None, h if pre else None
    check(lib().moe_norm_forward(plan[1], x.data_ptr(), _ptr(f), _ptr(gate), _ptr(w_post), _ptr(w_pre), _ptr(z),
                                 _ptr(h), _ptr(r_post), _ptr(r_pre), _stream(None)))
    return z, h, r_post, r_pre


def norm_backward(dz, dh, z, f=None, gate=None, w_post=None, w_pre=None, r_post=None, r_pre=None, *, gate_kind="none",
                  post=True, pre=True, alpha=1.0, need_dx=True, need_df=True, need_dgate=True, need_dw=True,
                  stream=None):
    """(dx, df, dgate, dw_post, dw_pre) of norm_forward from the gradients dz
    (None: nothing but h is used) and dh, its z, f and reciprocal roots; what
    does not exist or is not needed comes back as None."""
    if stream is not None:
        return _on(stream, norm_backward, dz, dh, z, f, gate, w_post, w_pre, r_post, r_pre, gate_kind=gate_kind, post=post,
                   pre=pre, alpha=alpha, need_dx=need_dx, need_df=need_df, need_dgate=need_dgate, need_dw=need_dw)
    like = dz if dz is not None else dh
    if not (like is not None and like.dim() == 2 and like.dtype in _ELEM):
        _bad("dz or dh must be a bf16, fp16 or fp32 matrix")
    rows, d = like.shape
    dt, dev, gpu, post = like.dtype, like.device, _gpu(like, "dz or dh"), post and f is not None
    if not (pre or dz is not None):
        _bad("without the pre norm the gradient arrives in dz")
    ld_z, ld_h, ld_f = d, d, d
    if dz is not None:
        dz, ld_z = _rows(dz, "dz", d, gpu, dt, rows)
    if pre:
        if not (dh is not None and z is not None and r_pre is not None):
            _bad("the pre norm needs dh, z and r_pre")
        dh, ld_h = _rows(dh, "dh", d, gpu, dt, rows)
        z, ld = _rows(z, "z", d, gpu, dt, rows)
        if dz is not None and ld != ld_z and rows > 1:      # the library has one stride for the two
            dz, z, ld = dz.contiguous(), z.contiguous(), d
        ld_z = ld
        r_pre = _vector(r_pre, "r_pre", rows, torch.float32, gpu)
    if f is not None:
        f, ld_f = _rows(f, "f", d, gpu, dt, rows)
    if post:
        if not (r_post is not None):
            _bad("the post norm needs r_post")
        r_post = _vector(r_post, "r_post", rows, torch.float32, gpu)
    gate, ld_g = _gate(gate, gate_kind, rows, d, dt, gpu)
    w_post = _vector(w_post, "w_post", d, dt, gpu) if post else None
    w_pre = _vector(w_pre, "w_pre", d, dt, gpu) if pre else None

    dx = torch.empty((rows, d), dtype=dt, device=dev) if need_dx else None
    df = dgate = None
    if f is not None and need_df:
        f, ld_f = _narrow(f, ld_f)
        df = torch.empty((rows, ld_f), dtype=dt, device=dev)
        if ld_f != d:
            df = df[:, :d]
    if gate is not None and need_dgate:
        if gate_kind == "full":
            gate, ld_g = _narrow(gate, ld_g)
        dgate = torch.empty((rows, ld_g), dtype=dt, device=dev)[:, :d] if gate_kind == "full" and ld_g != d else \
            torch.empty_like(gate)
    dw_post = torch.empty_like(w_post) if need_dw and w_post is not None else None
    dw_pre = torch.empty_like(w_pre) if need_dw and w_pre is not None else None
    plan = _norm_plan(rows, d, _ELEM[dt], (MOE_NORM_POST if post else 0) | (MOE_NORM_PRE if pre else 0),
                      GATES[gate_kind], float(alpha), 0.0, d, ld_f, ld_z, ld_h, ld_g)
    ws = _ws(plan, dev)
    check(lib().moe_norm_backward(plan[1], _ptr(dz), _ptr(dh), _ptr(z), _ptr(f), _ptr(gate), _ptr(w_post),
                                  _ptr(w_pre), _ptr(r_post), _ptr(r_pre), _ptr(dx), _ptr(df), _ptr(dgate),
                                  _ptr(dw_post), _ptr(dw_pre), ws.data_ptr(), _stream(None)))
    return dx, df, dgate, dw_post, dw_pre


# ---------------------------------------------------------------- embedding
@lru_cache(maxsize=512)
def _embed_plan(*fields):
    return _plan(MoeEmbedConfig(*fields), lib().moe_embed_workspace_bytes)


def _ids(ids, gpu, name="ids"):
    if not (ids.dtype in (torch.int32, torch.int64) and ids.get_device() == gpu):
        _bad("%s must be int32 or int64 on GPU %d", name, gpu)
    return ids if ids.dim() == 1 and ids.is_contiguous() else ids.reshape(-1).contiguous()


def embed_forward(ids, table, *, scale=1.0, out=None, stream=None):
    """scale * table[ids] [*ids.shape, d]; an id outside [0, V) (padding) gives a
    zero row.  table [V, d] bf16, fp16 or fp32; ids int32 or int64 of any shape.
    `out` [ids.numel(), d] may be given."""
    if stream is not None:
        return _on(stream, embed_forward, ids, table, scale=scale, out=out)
    if not (table.dim() == 2 and table.dtype in _ELEM):
        _bad("table must be a bf16, fp16 or fp32 matrix [V, d]")
    V, d = table.shape
    gpu = _gpu(table, "table")
    table, ld_t = _rows(table, "table", d, gpu)
    flat = _ids(ids, gpu)
    rows, el = flat.shape[0], _ELEM[table.dtype]
    res, ld_o = _out(out, "out", rows, d, table.dtype, table.device, gpu)
    plan = _embed_plan(rows, V, d, el, el, int(flat.dtype == torch.int64), 0, float(scale), ld_t, ld_o)
    check(lib().moe_embed_forward(plan[1], flat.data_ptr(), table.data_ptr(), res.data_ptr(), _stream(None)))
    return res if out is not None or ids.dim() == 1 else res.view(*ids.shape, d)


def embed_backward(ids, dout, V, *, scale=1.0, dtable=None, grad_dtype=None, accumulate=False, stream=None):
    """dtable [V, d]: dtable[v] = scale * sum of dout[t] over ids[t] = v, in
    ascending t.  dout [ids.numel(), d] (or [*ids.shape, d]); dtable of dout's
    type or fp32 (grad_dtype, or dtable's).  accumulate adds to the given
    dtable's rows that occur and leaves the others alone."""
    if stream is not None:
        return _on(stream, embed_backward, ids, dout, V, scale=scale, dtable=dtable, grad_dtype=grad_dtype,
                   accumulate=accumulate)
    gpu = _gpu(dout, "dout")
    flat = _ids(ids, gpu)
    if not (dout.dtype in _ELEM and dout.dim() >= min(2, 1 + ids.dim())):
        _bad("dout must be bf16, fp16 or fp32 [rows, d]")
    d = dout.shape[-1]
    if dout.dim() != 2:
        dout = dout.reshape(-1, d)
    dout, ld_o = _rows(dout, "dout", d, gpu, None, flat.shape[0])
    if not (not accumulate or dtable is not None):
        _bad("accumulate adds to a given dtable")
    grad_dtype = grad_dtype or (dtable.dtype if dtable is not None else dout.dtype)
    if not (grad_dtype in (dout.dtype, torch.float32)):
        _bad("dtable is of dout's type or float32")
    dtable, ld_t = _out(dtable, "dtable", V, d, grad_dtype, dout.device, gpu)
    plan = _embed_plan(flat.shape[0], V, d, _ELEM[dout.dtype], _ELEM[grad_dtype], int(flat.dtype == torch.int64),
                       int(accumulate), float(scale), ld_t, ld_o)
    ws = _ws(plan, dout.device)
    check(lib().moe_embed_backward(plan[1], flat.data_ptr(), dout.data_ptr(), dtable.data_ptr(), ws.data_ptr(),
                                   _stream(None)))
    if accumulate:
        _changed(dtable)
    return dtable


# ---------------------------------------------------------------- loss over a vocabulary
@lru_cache(maxsize=512)
def _vocab_plan(backward, *fields):
    return _plan(MoeVocabConfig(*fields), lib().moe_vocab_backward_workspace_bytes if backward
                 else lib().moe_vocab_forward_workspace_bytes)


def _vocab(x, w, labels):
    if not (x.dim() == 2 and x.dtype in (torch.bfloat16, torch.float16)):
        _bad("x must be a bf16 or fp16 matrix [rows, d]")
    gpu, (rows, d) = _gpu(x, "x"), x.shape
    if w.dim() != 2:
        _bad("w must be a matrix [V, %d]", d)
    x, ld_x = _rows(x, "x", d, gpu)
    w, ld_w = _rows(w, "w", d, gpu, x.dtype)
    flat = _ids(labels, gpu, "labels")
    if flat.shape[0] != rows:
        _bad("labels has %d entries, expected %d", flat.shape[0], rows)
    # TMA takes rows that start on 16-byte boundaries: others are copied in the call
    copy_w = int(ld_w % 8 != 0 or w.data_ptr() % 16 != 0)
    return gpu, x, ld_x, w, ld_w, flat, rows, w.shape[0], d, copy_w


def _per_row(t, name, rows, gpu, device):
    if t is None:
        return torch.empty(rows, dtype=torch.float32, device=device)
    if not (t.shape == (rows,) and t.dtype == torch.float32 and t.get_device() == gpu and t.is_contiguous()):
        _bad("%s must be a contiguous float32 vector of %d on GPU %d", name, rows, gpu)
    return t


def vocab_loss_forward(x, w, labels, *, loss=None, lse=None, return_workspace=False, stream=None):
    """(loss [rows], lse [rows]) fp32 of the logits z = x w^T, which are never in memory:
    lse[t] = log sum_v exp z[t, v], loss[t] = lse[t] - z[t, labels[t]].  x [rows, d]
    and w [V, d] bf16 or fp16, labels int32 or int64 of rows entries; a row whose
    label lies outside [0, V) (padding) does not count: both are zero, whatever x
    holds there."""
    if stream is not None:
        return _on(stream, vocab_loss_forward, x, w, labels, loss=loss, lse=lse, return_workspace=return_workspace)
    gpu, x, ld_x, w, ld_w, flat, rows, V, d, copy_w = _vocab(x, w, labels)
    loss, lse = _per_row(loss, "loss", rows, gpu, x.device), _per_row(lse, "lse", rows, gpu, x.device)
    el = _ELEM[x.dtype]
    plan = _vocab_plan(False, rows, V, d, el, el, int(flat.dtype == torch.int64), 0, copy_w, ld_x, ld_w, 0)
    ws = _ws(plan, x.device)
    check(lib().moe_vocab_forward(plan[1], x.data_ptr(), w.data_ptr(), flat.data_ptr(), loss.data_ptr(), lse.data_ptr(),
                                  ws.data_ptr(), _stream(None)))
    return (loss, lse, ws) if return_workspace else (loss, lse)


def vocab_loss_backward(dloss, x, w, labels, lse, *, dlse=None, dx=None, dw=None, need_dx=True, need_dw=True,
                        dw_dtype=None, accumulate=False, return_workspace=False, stream=None):
    """(dx [rows, d], dw [V, d]) of vocab_loss_forward from the gradients dloss and dlse
    [rows] fp32 of its two results (either may be None) and its lse; either output is
    None when not needed.  A row that does not count, or whose gradients are both zero,
    gets dx = 0 and adds nothing to dw.  dw is of x's type or fp32 (dw_dtype, or dw's);
    with accumulate it must be given, fp32, and is added to."""
    if stream is not None:
        return _on(stream, vocab_loss_backward, dloss, x, w, labels, lse, dlse=dlse, dx=dx, dw=dw, need_dx=need_dx,
                   need_dw=need_dw, dw_dtype=dw_dtype, accumulate=accumulate, return_workspace=return_workspace)
    gpu, x, ld_x, w, ld_w, flat, rows, V, d, copy_w = _vocab(x, w, labels)
    if dloss is None and dlse is None:
        _bad("the gradient arrives in dloss, dlse or both")
    dloss, dlse = _vector(dloss, "dloss", rows, torch.float32, gpu), _vector(dlse, "dlse", rows, torch.float32, gpu)
    lse = _vector(lse, "lse", rows, torch.float32, gpu)
    if lse is None:
        _bad("the backward needs the forward's lse")
    dw_dtype = dw_dtype or (dw.dtype if dw is not None else x.dtype)
    if not (dw_dtype in (x.dtype, torch.float32)):
        _bad("dw is of x's type or float32")
    if not (not accumulate or (dw is not None and dw_dtype == torch.float32)):
        _bad("accumulate adds to a given float32 dw")
    if not (need_dx or need_dw):
        _bad("nothing to compute")
    ld_dx = 0
    if need_dx:
        dx, ld_dx = _out(dx, "dx", rows, d, x.dtype, x.device, gpu)
    if need_dw:
        if dw is None:
            dw = torch.empty((V, d), dtype=dw_dtype, device=x.device)
        if not (dw.shape == (V, d) and dw.dtype == dw_dtype and dw.get_device() == gpu and dw.is_contiguous()):
            _bad("dw must be a contiguous %s matrix [%d, %d] on GPU %d", dw_dtype, V, d, gpu)
    plan = _vocab_plan(True, rows, V, d, _ELEM[x.dtype], _ELEM[dw_dtype], int(flat.dtype == torch.int64), int(accumulate),
                       copy_w, ld_x, ld_w, ld_dx)
    ws = _ws(plan, x.device)
    dx, dw = dx if need_dx else None, dw if need_dw else None
    check(lib().moe_vocab_backward(plan[1], _ptr(dloss), _ptr(dlse), x.data_ptr(), w.data_ptr(), flat.data_ptr(),
                                   lse.data_ptr(), _ptr(dx), _ptr(dw), ws.data_ptr(), _stream(None)))
    if accumulate and need_dw:
        _changed(dw)
    return (dx, dw, ws) if return_workspace else (dx, dw)


# ---------------------------------------------------------------- all gradients
def _dense(t):
    """Whether t's elements fill its memory, in whatever order of dimensions."""
    if t.is_contiguous():
        return True
    order = sorted(range(t.dim()), key=lambda i: (t.stride(i), t.shape[i]), reverse=True)
    return t.permute(order).is_contiguous()


_device_of, _is_contiguous, _numel, _address = (torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.numel,
                                                torch.Tensor.data_ptr)
_type_of, _shape_of, _strides_of = attrgetter("dtype"), attrgetter("shape"), torch.Tensor.stride


def _tensors(ts, gpu, name):
    """(types, counts, addresses) of dense tensors on the current GPU, as host arrays.  By
    map over the methods: 400 tensors take half of what a loop over them does."""
    if ts and set(map(_device_of, ts)) != {gpu}:
        _bad("%s are not all on the current GPU", name)
    if not all(map(_is_contiguous, ts)):
        for t in ts:
            if not _dense(t):
                _bad("one of %s (shape %s, strides %s) does not fill its memory", name, tuple(t.shape), t.stride())
    types = list(map(_ELEM.get, map(_type_of, ts)))
    if None in types:
        _bad("%s are bf16, fp16 or fp32", name)
    return array("i", types), array("q", list(map(_numel, ts))), array("Q", list(map(_address, ts)))


def _host(a):
    return a.buffer_info()[0] if len(a) else None


@lru_cache(maxsize=512)
def _grad_workspace(n):
    return lib().moe_grad_workspace_bytes(n)


def _norm_out(norm, gpu):
    if norm is None:
        return torch.empty((), dtype=torch.float32, device=torch.device("cuda", gpu))
    if not (norm.numel() == 1 and norm.dtype == torch.float32 and norm.get_device() == gpu):
        _bad("norm must be one float32 on GPU %d", gpu)
    return norm


def grad_norm(grads, *, norm=None, stream=None):
    """The 2-norm of all elements of the tensors in the list `grads` (bf16, fp16 or fp32,
    any mix; each fills its memory): a 0-d fp32 tensor, zero for no tensors."""
    if stream is not None:
        return _on(stream, grad_norm, list(grads), norm=norm)
    grads, gpu = list(grads), _current_gpu()
    types, counts, at = _tensors(grads, gpu, "grads")
    norm = _norm_out(norm, gpu)
    ws = torch.empty(_grad_workspace(len(grads)), dtype=torch.uint8, device=norm.device)
    check(lib().moe_grad_norm(_host(at), _host(counts), _host(types), len(grads), norm.data_ptr(), ws.data_ptr(),
                              _stream(None)))
    return norm


def grad_clip(grads, max_norm, *, out=None, eps=1e-6, norm=None, stream=None):
    """Scales all tensors of the list `grads` by min(1, max_norm / (norm + eps)), in place
    or into the list `out` of tensors of the same shapes and layouts (each of its
    gradient's type or fp32, as an optimizer's masters take them); the norm of before
    comes back as a 0-d fp32 tensor.  An infinite max_norm is no limit, whatever the norm
    but NaN.  No output shares memory with another tensor of the
    call (the same gradient twice, a view of another): refused."""
    if stream is not None:
        return _on(stream, grad_clip, list(grads), max_norm, out=None if out is None else list(out), eps=eps, norm=norm)
    grads, gpu = list(grads), _current_gpu()
    types, counts, at = _tensors(grads, gpu, "grads")
    out_types, out_at = types, at
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            _bad("out has %d tensors, expected %d", len(out), len(grads))
        out_types, _, out_at = _tensors(out, gpu, "out")
        same = list(map(_shape_of, grads)) == list(map(_shape_of, out))
        if same and list(map(_strides_of, grads)) != list(map(_strides_of, out)):
            same = all(g.stride() == o.stride() or (g.is_contiguous() and o.is_contiguous()) for g, o in zip(grads, out))
        if not same or any(o != t and o != MOE_ELEM_FP32 for t, o in zip(types, out_types)):
            _bad("out's tensors have their gradients' shapes and layouts, and their types or float32")
    max_norm, eps = float(max_norm), float(eps)
    if not (max_norm >= 0.0 and 0.0 < eps < float("inf")):
        _bad("max_norm must not be negative, eps must be positive")
    norm = _norm_out(norm, gpu)
    ws = torch.empty(_grad_workspace(len(grads)), dtype=torch.uint8, device=norm.device)
    rc = lib().moe_grad_clip(ctypes.byref(MoeClipConfig(max_norm, eps)), _host(at), _host(out_at), _host(counts),
                             _host(types), _host(out_types), len(grads), norm.data_ptr(), ws.data_ptr(), _stream(None))
    if rc == -1:    # of the library's checks the only one that is not made above
        _bad("tensors of the call overlap: no output shares memory with another tensor")
    check(rc)
    _changed(grads if out is None else out)
    return norm
