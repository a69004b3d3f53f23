"""CPU-only checks of the entry points around the layer: argument checks of the
library and of block.py, sizes of the workspaces.  No compute call is made."""
import ctypes

import pytest
import torch

P = 1 << 12     # an aligned pointer that is never followed


@pytest.fixture(scope="module")
def pkg():
    from mixture_experts_layer_device_gb300 import build
    build.build()
    import mixture_experts_layer_device_gb300 as m
    return m


def grouped(pkg, **kw):
    a = dict(rows=10, E=3, N=16, K=24, dtype=0, out_dtype=0, accumulate=0, ld_x=0, ld_y=0, ld_w=0, ld_e=0)
    a.update(kw)
    return pkg.MoeGroupedConfig(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), -1), (dict(E=0), -1), (dict(N=0), -1), (dict(K=-3), -1), (dict(dtype=2), -1), (dict(dtype=7), -1),
    (dict(out_dtype=1), -1), (dict(accumulate=1), -1), (dict(accumulate=2, out_dtype=2), -1), (dict(E=32768), -2),
    (dict(N=(1 << 20) + 1), -2), (dict(rows=1 << 31), -2), (dict(ld_x=23), -2), (dict(ld_y=15), -2), (dict(ld_w=8), -2),
    (dict(ld_x=1 << 31), -2), (dict(ld_x=-24), -2), (dict(ld_e=16 * 24 - 1), -2), (dict(ld_w=32, ld_e=16 * 24), -2)])
def test_grouped_refusals(pkg, bad, code):
    cfg = grouped(pkg, **bad)
    assert pkg.moe_grouped_workspace_bytes(cfg) == 0
    assert pkg.moe_grouped_forward(cfg, P, P, P, P, P, 0) == code
    assert pkg.moe_grouped_backward(cfg, P, P, P, P, P, P, P, 0) == code


def test_grouped_pointers(pkg):
    cfg = grouped(pkg)
    assert pkg.moe_grouped_workspace_bytes(cfg) >= 256 + 4 * 4
    for i in range(5):
        a = [P] * 5
        a[i] = None
        assert pkg.moe_grouped_forward(cfg, *a, 0) == -1
        a[i] = P + 1
        assert pkg.moe_grouped_forward(cfg, *a, 0) == -3
    assert pkg.moe_grouped_forward(grouped(pkg, out_dtype=2), P, P, P, P + 2, P, 0) == -3
    assert pkg.moe_grouped_forward(grouped(pkg, out_dtype=2, accumulate=1), P, P, P, P, P, 0) == -1
    assert pkg.moe_grouped_backward(cfg, P, P, P, P, None, None, P, 0) == -1    # nothing to write
    assert pkg.moe_grouped_backward(cfg, P, None, P, P, P, P, P, 0) == -1       # dw needs x
    assert pkg.moe_grouped_backward(cfg, P, P, None, P, P, P, P, 0) == -1       # dx needs w
    assert pkg.moe_grouped_backward(cfg, P, P, P, P + 2, P, P, P, 0) == -3
    assert pkg.lib().moe_grouped_forward(None, P, P, P, P, P, None) == -1


def norm(pkg, **kw):
    a = dict(rows=4, d=64, dtype=0, flags=3, gate=0, alpha=1.0, eps=1e-6, ld_x=0, ld_f=0, ld_z=0, ld_h=0, ld_g=0)
    a.update(kw)
    return pkg.MoeNormConfig(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), -1), (dict(d=0), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(flags=4), -1), (dict(gate=4), -1),
    (dict(gate=-1), -1), (dict(alpha=float("nan")), -1), (dict(alpha=float("inf")), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1), (dict(d=65537), -2), (dict(rows=1 << 31), -2), (dict(ld_x=63), -2), (dict(ld_f=1), -2),
    (dict(ld_z=-64), -2), (dict(ld_h=1 << 31), -2), (dict(ld_g=63), -2)])
def test_norm_refusals(pkg, bad, code):
    cfg = norm(pkg, **bad)
    assert pkg.moe_norm_workspace_bytes(cfg) == 0
    assert pkg.moe_norm_forward(cfg, *[P] * 9, 0) == code
    assert pkg.moe_norm_backward(cfg, *[P] * 15, 0) == code


def test_norm_pointers(pkg):
    ok = [P] * 9        # x f gate w_post w_pre z h r_post r_pre
    def fwd(cfg, **kw):
        a = dict(zip(("x", "f", "gate", "w_post", "w_pre", "z", "h", "r_post", "r_pre"), ok))
        a.update(kw)
        return pkg.moe_norm_forward(cfg, *a.values(), 0)
    assert fwd(norm(pkg), x=None) == -1 and fwd(norm(pkg), f=None) == -1 and fwd(norm(pkg), h=None) == -1
    assert fwd(norm(pkg, flags=1), z=None) == -1
    assert fwd(norm(pkg, flags=0, gate=1), f=None) == -1 and fwd(norm(pkg, gate=2), gate=None) == -1
    assert fwd(norm(pkg), z=P + 1) == -3 and fwd(norm(pkg, dtype=2), w_pre=P + 2) == -3
    assert fwd(norm(pkg), r_post=P + 2) == -3
    names = ("dz", "dh", "z", "f", "gate", "w_post", "w_pre", "r_post", "r_pre", "dx", "df", "dgate", "dw_post", "dw_pre", "ws")
    def bwd(cfg, **kw):
        a = dict.fromkeys(names, P)
        a.update(dict(dgate=None) if cfg.gate == 0 else {}, **kw)
        return pkg.moe_norm_backward(cfg, *a.values(), 0)
    assert bwd(norm(pkg), dgate=P) == -1                       # no gate, no gradient of one
    assert bwd(norm(pkg, flags=2)) == -1                       # dw_post without the post norm
    assert bwd(norm(pkg, flags=1)) == -1                       # dw_pre without the pre norm
    assert bwd(norm(pkg, flags=1), dw_pre=None, dz=None) == -1
    for miss in ("dh", "z", "r_pre", "f", "r_post", "ws"):
        assert bwd(norm(pkg), **{miss: None}) == -1, miss
    assert bwd(norm(pkg, gate=1), gate=None) == -1
    assert bwd(norm(pkg), dx=P + 1) == -3 and bwd(norm(pkg), ws=P + 8) == -3 and bwd(norm(pkg), r_pre=P + 1) == -3


def embed(pkg, **kw):
    a = dict(rows=4, V=10, d=16, dtype=0, grad_dtype=0, ids64=1, accumulate=0, scale=1.0, ld_t=0, ld_o=0)
    a.update(kw)
    return pkg.MoeEmbedConfig(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), -1), (dict(V=0), -1), (dict(d=0), -1), (dict(dtype=3), -1), (dict(grad_dtype=1), -1),
    (dict(dtype=2, grad_dtype=0), -1), (dict(ids64=2), -1), (dict(accumulate=-1), -1), (dict(scale=float("nan")), -1),
    (dict(rows=1 << 30), -2), (dict(V=(1 << 31) - 1), -2), (dict(d=(1 << 20) + 1), -2), (dict(ld_t=15), -2),
    (dict(ld_o=1 << 31), -2)])
def test_embedding_refusals(pkg, bad, code):
    cfg = embed(pkg, **bad)
    assert pkg.moe_embed_workspace_bytes(cfg) == 0
    assert pkg.moe_embed_forward(cfg, P, P, P, 0) == code
    assert pkg.moe_embed_backward(cfg, P, P, P, P, 0) == code


def test_embedding_pointers_and_workspace(pkg):
    cfg = embed(pkg)
    for i in range(3):
        a = [P] * 3
        a[i] = None
        assert pkg.moe_embed_forward(cfg, *a, 0) == -1
        a[i] = P + 1
        assert pkg.moe_embed_forward(cfg, *a, 0) == -3
    assert pkg.moe_embed_forward(cfg, P + 4, P, P, 0) == -3                     # int64 ids
    assert pkg.moe_embed_backward(cfg, P, P, P, None, 0) == -1
    assert pkg.moe_embed_backward(cfg, P, P, P, P + 8, 0) == -3
    assert pkg.moe_embed_workspace_bytes(embed(pkg, rows=0)) > 0
    assert pkg.moe_embed_workspace_bytes(embed(pkg, rows=1 << 20, V=1 << 17)) >= (1 << 20) * 16 + (1 << 17)


def test_python_functions_check_before_they_call(pkg):
    """Shapes, types and places are refused with a ValueError; CPU tensors too."""
    from mixture_experts_layer_device_gb300 import block
    x, w, off = torch.zeros(4, 8), torch.zeros(2, 6, 8), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        block.grouped_forward(x, w, off)                                        # fp32
    with pytest.raises(ValueError):
        block.grouped_forward(x.bfloat16(), w.bfloat16(), off)                  # not on the GPU
    with pytest.raises(ValueError):
        block.grouped_backward(x.bfloat16(), x.bfloat16(), w.half(), off)
    with pytest.raises(ValueError):
        block.norm_forward(x.double())
    with pytest.raises(ValueError):
        block.norm_forward(x, x, x, gate_kind="none")
    with pytest.raises(ValueError):
        block.norm_backward(None, None, x)
    with pytest.raises(ValueError):
        block.embed_forward(off, x)
    with pytest.raises(ValueError):
        block.embed_backward(off.float(), x, 5)


def test_config_layouts_match_the_header(pkg):
    """The ctypes structures have the C structs' sizes (8-byte alignment)."""
    assert ctypes.sizeof(pkg.MoeGroupedConfig) == 8 + 6 * 4 + 4 * 8
    assert ctypes.sizeof(pkg.MoeNormConfig) == 8 + 4 * 4 + 2 * 4 + 5 * 8
    assert ctypes.sizeof(pkg.MoeEmbedConfig) == 16 + 6 * 4 + 2 * 8
