"""What a model needs around the MoE layer, on torch tensors: ragged matrix
products grouped by expert, the norms around a block with its gate and
residual scale, and the token embedding with its gradient (include/moe.h:
moe_grouped_*, moe_norm_*, moe_embed_*).

Plain functions: they check their arguments, allocate outputs and workspaces
from torch and call the library; all arithmetic runs in its kernels.  They run
on torch's current stream and do not synchronise; with `stream` (a stream or its
handle) they run as under `torch.cuda.stream(stream)`: what they read has to be
ready on it, and what they return is.  All tensors of a call are on the current
GPU.  The autograd functions and modules over them are in module.py.
"""
import ctypes
from functools import lru_cache

import torch

from . import (GATES, MOE_ELEM_BF16, MOE_ELEM_FP16, MOE_ELEM_FP32, MOE_NORM_POST, MOE_NORM_PRE, MoeEmbedConfig,
               MoeGroupedConfig, MoeNormConfig, _stream, check, lib, moe_get_status)

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
    for t in (*args, *kw.values()):
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
    dw_dtype = dw_dtype or (dw.dtype if dw is not None else dy.dtype)
    if not (dw_dtype in (dy.dtype, torch.float32)):
        _bad("dw is of dy's type or float32")
    if not (not accumulate or (dw is not None and dw_dtype == torch.float32)):
        _bad("accumulate adds to a given float32 dw")
    if not (need_dx or need_dw):
        _bad("nothing to compute")
    if need_dx:
        if dx is None:
            x, ld_x = _narrow(x, ld_x)
            dx = torch.empty((rows, ld_x), dtype=dy.dtype, device=dy.device)
            dx = dx if ld_x == K else dx[:, :K]
        if not (dx.shape == (rows, K) and dx.dtype == dy.dtype and dx.get_device() == gpu and
                (K == 1 or dx.stride(1) == 1)):
            _bad("dx must be a %s matrix [%d, %d] with contiguous rows on GPU %d", dy.dtype, rows, K, gpu)
        if rows > 1 and dx.stride(0) != ld_x:
            x, ld_x = x.contiguous(), K
            if not (dx.stride(0) == K):
                _bad("dx must have x's row stride or be contiguous")
    if need_dw:
        if dw is None:
            dw = torch.empty((E, N, K), dtype=dw_dtype, device=dy.device)
        if not (dw.shape == (E, N, K) and dw.dtype == dw_dtype and dw.get_device() == gpu and dw.is_contiguous()):
            _bad("dw must be a contiguous %s tensor [%d, %d, %d] on GPU %d", dw_dtype, E, N, K, gpu)
    ld_e = w.stride(0) if E > 1 else 0
    plan = _grouped_plan(rows, E, N, K, _ELEM[dy.dtype], _ELEM[dw_dtype], int(accumulate), ld_x, ld_y, ld_w, ld_e)
    ws = _ws(plan, dy.device)
    out = (dx if need_dx else None, dw if need_dw else None)
    check(lib().moe_grouped_backward(plan[1], dy.data_ptr(), x.data_ptr(), w.data_ptr(), offsets.data_ptr(),
                                     _ptr(out[0]), _ptr(out[1]), ws.data_ptr(), _stream(None)))
    return out + (ws,) if return_workspace else out


def grouped_status(ws, stream=None):
    """Synchronises the current stream, or `stream`: the one that the call ran on.  The
    device status of the call that used workspace `ws` (return_workspace=True): 0, or
    -7 when its offsets descend or leave the rows."""
    return moe_get_status(ws, stream)


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


def _ids(ids, gpu):
    if not (ids.dtype in (torch.int32, torch.int64) and ids.get_device() == gpu):
        _bad("ids must be int32 or int64 on GPU %d", gpu)
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
    return dtable
