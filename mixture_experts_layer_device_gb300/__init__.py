"""Python binding of the GB300 mixture-of-experts layer library (include/moe.h).

Argument marshalling only: every step of the layer runs in the CUDA kernels of
``libmoe_gb300.so``.  Functions take torch tensors (or raw device pointers as
ints, or None for NULL) and a stream (default: torch's current stream) and
return the library's status code; :func:`check` turns a non-zero code into an
exception.  There is no CPU fallback: importing the binding without the built
library raises.
"""
import ctypes
import os

from . import build as _build

# MOE_GB300_LIB names another build of the library (e.g. the bounds-checked
# debug build, build.build(debug=True)) for this process.
LIB_PATH = os.environ.get("MOE_GB300_LIB") or _build.LIB

MOE_BF16, MOE_MXFP8, MOE_NVFP4 = 0, 1, 2
DTYPES = {"bf16": MOE_BF16, "mxfp8": MOE_MXFP8, "nvfp4": MOE_NVFP4}
MOE_FLAG_BACKWARD = 1
MOE_FLAG_DEBUG_STARVE = 2
MOE_FLAG_DEBUG_DUMP = 4
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported shape", -3: "pointer not aligned as its entry point requires",
          -4: "CUDA error", -5: "device is not sm_103", -6: "a device-side wait timed out",
          -7: "a device-side bounds check failed: an index or offset out of range"}

MOE_ELEM_BF16, MOE_ELEM_FP16, MOE_ELEM_FP32 = 0, 1, 2
MOE_NORM_POST, MOE_NORM_PRE = 1, 2
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_ROW, MOE_GATE_FULL = 0, 1, 2, 3
GATES = {"none": MOE_GATE_NONE, "channel": MOE_GATE_CHANNEL, "row": MOE_GATE_ROW, "full": MOE_GATE_FULL}

WEIGHT_FIELDS = ["gu", "gu_scale", "dn", "dn_scale", "gu_t", "gu_t_scale", "dn_t", "dn_t_scale",
                 "s_gu", "s_dn", "s_gu_t", "s_dn_t", "gu_gscale", "dn_gscale"]


class MoeConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "d", "m", "E", "k", "m_shared", "dtype", "flags",
                                              "ring_rows", "gather_sms")] + [("aux_alpha", ctypes.c_float)]


class MoeWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in WEIGHT_FIELDS]


class MoeGroupedConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in ("E", "N", "K", "dtype", "out_dtype",
                                                                          "accumulate")] + \
               [(n, ctypes.c_int64) for n in ("ld_x", "ld_y", "ld_w", "ld_e")]


class MoeNormConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in ("d", "dtype", "flags", "gate")] + \
               [("alpha", ctypes.c_float), ("eps", ctypes.c_float)] + \
               [(n, ctypes.c_int64) for n in ("ld_x", "ld_f", "ld_z", "ld_h", "ld_g")]


class MoeEmbedConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("V", ctypes.c_int64)] + \
               [(n, ctypes.c_int32) for n in ("d", "dtype", "grad_dtype", "ids64", "accumulate")] + \
               [("scale", ctypes.c_float), ("ld_t", ctypes.c_int64), ("ld_o", ctypes.c_int64)]


_lib = None
EXPORTS = ["moe_workspace_bytes", "moe_saved_bytes", "moe_buffer_info", "moe_padded_rows",
           "moe_quantize_weights", "moe_quantize_mx", "moe_quantize_mx_both", "moe_prepare_weights",
           "moe_prepare_scales",
           "moe_canonical_scales", "moe_transpose_bf16", "moe_route",
           "moe_forward", "moe_backward",
           "moe_get_status", "moe_status_string", "moe_trace_enable", "moe_trace_clear", "moe_trace_count",
           "moe_trace_name", "moe_trace_ms", "moe_route_noalloc", "moe_router_forward", "moe_router_backward",
           "moe_grouped_workspace_bytes", "moe_grouped_forward", "moe_grouped_backward", "moe_norm_forward",
           "moe_norm_workspace_bytes", "moe_norm_backward", "moe_embed_forward", "moe_embed_workspace_bytes",
           "moe_embed_backward"]


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoe_gb300.so is not built (run __graft_entry__.build() or "
                               "python -m mixture_experts_layer_device_gb300.build)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
        cfgp = ctypes.POINTER(MoeConfig)
        L.moe_workspace_bytes.argtypes, L.moe_workspace_bytes.restype = [cfgp], Z
        L.moe_saved_bytes.argtypes, L.moe_saved_bytes.restype = [cfgp], Z
        L.moe_buffer_info.argtypes = [cfgp, I, ctypes.c_char_p, ctypes.POINTER(Z), ctypes.POINTER(Z)]
        L.moe_buffer_info.restype = I
        L.moe_padded_rows.argtypes, L.moe_padded_rows.restype = [cfgp], ctypes.c_int64
        L.moe_quantize_weights.argtypes, L.moe_quantize_weights.restype = [cfgp, P, I, I, I, P, P, S], I
        L.moe_quantize_mx.argtypes, L.moe_quantize_mx.restype = [P, I, I, I, I, P, P, S], I
        L.moe_quantize_mx_both.argtypes, L.moe_quantize_mx_both.restype = [P, I, I, I, P, P, P, P, S], I
        L.moe_prepare_weights.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, P, P, P, S]
        L.moe_prepare_weights.restype = I
        L.moe_prepare_scales.argtypes, L.moe_prepare_scales.restype = [P, ctypes.c_int64, ctypes.c_int32, P, S], I
        L.moe_canonical_scales.argtypes = [P, ctypes.c_int64, ctypes.c_int32, P, S]
        L.moe_canonical_scales.restype = I
        L.moe_transpose_bf16.argtypes, L.moe_transpose_bf16.restype = [P, I, I, I, P, S], I
        L.moe_route.argtypes, L.moe_route.restype = [cfgp, P, P, P, P, P, P, P, S], I
        L.moe_forward.argtypes = [cfgp, P, P, ctypes.POINTER(MoeWeights), P, P, P, S]
        L.moe_forward.restype = I
        L.moe_backward.argtypes = [cfgp, P, P, ctypes.POINTER(MoeWeights), P, P, P, P, P, P, P, P, S]
        L.moe_backward.restype = I
        L.moe_get_status.argtypes, L.moe_get_status.restype = [P, S], I
        L.moe_status_string.argtypes, L.moe_status_string.restype = [I], ctypes.c_char_p
        L.moe_route_noalloc.argtypes, L.moe_route_noalloc.restype = [cfgp, P, P, P, P, P, P, S], I
        L.moe_router_forward.argtypes, L.moe_router_forward.restype = [cfgp, P, P, P, P, S], I
        L.moe_router_backward.argtypes, L.moe_router_backward.restype = [cfgp, P, P, P, P, P, P, S], I
        L.moe_trace_enable.argtypes, L.moe_trace_enable.restype = [I], I
        L.moe_trace_clear.argtypes, L.moe_trace_clear.restype = [], None
        L.moe_trace_count.argtypes, L.moe_trace_count.restype = [], I
        L.moe_trace_name.argtypes, L.moe_trace_name.restype = [I], ctypes.c_char_p
        L.moe_trace_ms.argtypes, L.moe_trace_ms.restype = [I], ctypes.c_float
        gp, npp, ep = (ctypes.POINTER(c) for c in (MoeGroupedConfig, MoeNormConfig, MoeEmbedConfig))
        for fn, cp in ((L.moe_grouped_workspace_bytes, gp), (L.moe_norm_workspace_bytes, npp),
                       (L.moe_embed_workspace_bytes, ep)):
            fn.argtypes, fn.restype = [cp], Z
        for fn, cp, n in ((L.moe_grouped_forward, gp, 5), (L.moe_grouped_backward, gp, 7), (L.moe_norm_forward, npp, 9),
                          (L.moe_norm_backward, npp, 15), (L.moe_embed_forward, ep, 3),
                          (L.moe_embed_backward, ep, 4)):
            fn.argtypes, fn.restype = [cp] + [P] * n + [S], I
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current_stream = None


def _stream(stream):
    global _current_stream
    if stream is None:
        if _current_stream is None:
            import torch
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # the same handle, without the Stream object
            device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
            _current_stream = (lambda: raw(device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def config(T, d, m, E, k, m_shared=0, dtype=MOE_BF16, flags=0, ring_rows=0, gather_sms=0, aux_alpha=0.0):
    if isinstance(dtype, str):
        dtype = DTYPES[dtype]
    return MoeConfig(T, d, m, E, k, m_shared, dtype, flags, ring_rows, gather_sms, aux_alpha)


def moe_router_forward(cfg, x, W_r, logits, ws, stream=None):
    return lib().moe_router_forward(ctypes.byref(cfg), _ptr(x), _ptr(W_r), _ptr(logits), _ptr(ws), _stream(stream))


def moe_router_backward(cfg, dlogits, x, W_r, dx, dW_r, ws, stream=None):
    return lib().moe_router_backward(ctypes.byref(cfg), _ptr(dlogits), _ptr(x), _ptr(W_r), _ptr(dx), _ptr(dW_r),
                                     _ptr(ws), _stream(stream))


def weights(**kw):
    """MoeWeights from keyword tensors (names as in moe_weights)."""
    w = MoeWeights()
    for n in WEIGHT_FIELDS:
        setattr(w, n, _ptr(kw.get(n)))
    return w


def check(rc):
    if rc != 0:
        raise RuntimeError("moe library error %d: %s" % (rc, STATUS.get(rc, "unknown")))
    return rc


def moe_workspace_bytes(cfg):
    return lib().moe_workspace_bytes(ctypes.byref(cfg))


def moe_saved_bytes(cfg):
    return lib().moe_saved_bytes(ctypes.byref(cfg))


def moe_padded_rows(cfg):
    return lib().moe_padded_rows(ctypes.byref(cfg))


def moe_buffer_info(cfg, which, name):
    off, nb = ctypes.c_size_t(), ctypes.c_size_t()
    check(lib().moe_buffer_info(ctypes.byref(cfg), which, name.encode(), ctypes.byref(off), ctypes.byref(nb)))
    return off.value, nb.value


def moe_quantize_mx_both(src, batch, rows, cols, codes, scales, codes_t, scales_t, stream=None):
    return lib().moe_quantize_mx_both(_ptr(src), batch, rows, cols, _ptr(codes), _ptr(scales), _ptr(codes_t),
                                      _ptr(scales_t), _stream(stream))


def moe_quantize_weights(cfg, w_bf16, rows, cols, blocks_along_rows, codes, scales, stream=None):
    return lib().moe_quantize_weights(ctypes.byref(cfg), _ptr(w_bf16), rows, cols, int(blocks_along_rows),
                                      _ptr(codes), _ptr(scales), _stream(stream))


def moe_quantize_mx(src, batch, rows, cols, transpose, codes, scales, stream=None):
    return lib().moe_quantize_mx(_ptr(src), batch, rows, cols, int(transpose), _ptr(codes), _ptr(scales),
                                 _stream(stream))


def moe_prepare_weights(cfg, w_gu, w_dn, gu, gu_scale, dn, dn_scale, gu_t=None, gu_t_scale=None, dn_t=None,
                        dn_t_scale=None, gu_gscale=None, dn_gscale=None, stream=None):
    return lib().moe_prepare_weights(ctypes.byref(cfg), _ptr(w_gu), _ptr(w_dn), _ptr(gu), _ptr(gu_scale), _ptr(dn),
                                     _ptr(dn_scale), _ptr(gu_t), _ptr(gu_t_scale), _ptr(dn_t), _ptr(dn_t_scale),
                                     _ptr(gu_gscale), _ptr(dn_gscale), _stream(stream))


def moe_prepare_scales(scales, rows, K, prepared, stream=None):
    return lib().moe_prepare_scales(_ptr(scales), rows, K, _ptr(prepared), _stream(stream))


def moe_canonical_scales(prepared, rows, K, scales, stream=None):
    return lib().moe_canonical_scales(_ptr(prepared), rows, K, _ptr(scales), _stream(stream))


def moe_transpose_bf16(src, batch, rows, cols, dst, stream=None):
    return lib().moe_transpose_bf16(_ptr(src), batch, rows, cols, _ptr(dst), _stream(stream))


def moe_route(cfg, logits, idx, w, counts, offsets, perm, ws, stream=None):
    return lib().moe_route(ctypes.byref(cfg), _ptr(logits), _ptr(idx), _ptr(w), _ptr(counts), _ptr(offsets),
                           _ptr(perm), _ptr(ws), _stream(stream))


def moe_route_noalloc(cfg, logits, idx, w, counts, offsets, perm, stream=None):
    return lib().moe_route_noalloc(ctypes.byref(cfg), _ptr(logits), _ptr(idx), _ptr(w), _ptr(counts),
                                   _ptr(offsets), _ptr(perm), _stream(stream))


def moe_forward(cfg, x, logits, W, y, saved, ws, stream=None):
    return lib().moe_forward(ctypes.byref(cfg), _ptr(x), _ptr(logits), ctypes.byref(W), _ptr(y), _ptr(saved),
                             _ptr(ws), _stream(stream))


def moe_backward(cfg, dy, x, W, saved, dx, dlogits, dW_gu, dW_dn, dWs_gu, dWs_dn, ws, stream=None):
    return lib().moe_backward(ctypes.byref(cfg), _ptr(dy), _ptr(x), ctypes.byref(W), _ptr(saved), _ptr(dx),
                              _ptr(dlogits), _ptr(dW_gu), _ptr(dW_dn), _ptr(dWs_gu), _ptr(dWs_dn), _ptr(ws),
                              _stream(stream))


def moe_grouped_workspace_bytes(cfg):
    return lib().moe_grouped_workspace_bytes(ctypes.byref(cfg))


def moe_grouped_forward(cfg, x, w, offsets, y, ws, stream=None):
    return lib().moe_grouped_forward(ctypes.byref(cfg), _ptr(x), _ptr(w), _ptr(offsets), _ptr(y), _ptr(ws),
                                     _stream(stream))


def moe_grouped_backward(cfg, dy, x, w, offsets, dx, dw, ws, stream=None):
    return lib().moe_grouped_backward(ctypes.byref(cfg), _ptr(dy), _ptr(x), _ptr(w), _ptr(offsets), _ptr(dx),
                                      _ptr(dw), _ptr(ws), _stream(stream))


def moe_norm_forward(cfg, x, f, gate, w_post, w_pre, z, h, r_post, r_pre, stream=None):
    return lib().moe_norm_forward(ctypes.byref(cfg), _ptr(x), _ptr(f), _ptr(gate), _ptr(w_post), _ptr(w_pre),
                                  _ptr(z), _ptr(h), _ptr(r_post), _ptr(r_pre), _stream(stream))


def moe_norm_workspace_bytes(cfg):
    return lib().moe_norm_workspace_bytes(ctypes.byref(cfg))


def moe_norm_backward(cfg, dz, dh, z, f, gate, w_post, w_pre, r_post, r_pre, dx, df, dgate, dw_post, dw_pre, ws,
                      stream=None):
    return lib().moe_norm_backward(ctypes.byref(cfg), _ptr(dz), _ptr(dh), _ptr(z), _ptr(f), _ptr(gate),
                                   _ptr(w_post), _ptr(w_pre), _ptr(r_post), _ptr(r_pre), _ptr(dx), _ptr(df),
                                   _ptr(dgate), _ptr(dw_post), _ptr(dw_pre), _ptr(ws), _stream(stream))


def moe_embed_forward(cfg, ids, table, out, stream=None):
    return lib().moe_embed_forward(ctypes.byref(cfg), _ptr(ids), _ptr(table), _ptr(out), _stream(stream))


def moe_embed_workspace_bytes(cfg):
    return lib().moe_embed_workspace_bytes(ctypes.byref(cfg))


def moe_embed_backward(cfg, ids, dout, dtable, ws, stream=None):
    return lib().moe_embed_backward(ctypes.byref(cfg), _ptr(ids), _ptr(dout), _ptr(dtable), _ptr(ws),
                                    _stream(stream))


def moe_get_status(ws, stream=None):
    return lib().moe_get_status(_ptr(ws), _stream(stream))


def moe_trace_enable(capacity):
    return lib().moe_trace_enable(capacity)


def moe_trace_clear():
    lib().moe_trace_clear()


def moe_trace_records():
    """[(kernel name, milliseconds)] of the launches recorded since the last clear."""
    L = lib()
    return [(L.moe_trace_name(i).decode(), L.moe_trace_ms(i)) for i in range(L.moe_trace_count())]
