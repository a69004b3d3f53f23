"""CPU-only checks of the entry points that end a training step: argument checks of
the library and of block.py, sizes of the workspaces.  No compute call is made."""
import ctypes
from array import array

import pytest
import torch

P = 1 << 12     # an aligned pointer that is never followed


@pytest.fixture(scope="module")
def pkg():
    from mixture_experts_layer_device_gb300 import build
    build.build()
    import mixture_experts_layer_device_gb300 as m
    return m


def gated(pkg, **kw):
    a = dict(rows=10, E=3, m=8, K=24, dtype=0, grad_dtype=0, act=0, accumulate=0, ld_x=0, ld_h=0, ld_gu=0, ld_w=0, ld_e=0)
    a.update(kw)
    return pkg.MoeGatedConfig(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), -1), (dict(E=0), -1), (dict(m=0), -1), (dict(m=-4), -1), (dict(K=0), -1), (dict(dtype=2), -1),
    (dict(grad_dtype=1), -1), (dict(act=4), -1), (dict(act=-1), -1), (dict(accumulate=1), -1), (dict(accumulate=2), -1),
    (dict(E=32768), -2), (dict(m=(1 << 19) + 1), -2), (dict(m=1 << 30), -2), (dict(K=(1 << 20) + 1), -2),
    (dict(rows=1 << 31), -2), (dict(ld_x=23), -2), (dict(ld_h=7), -2), (dict(ld_gu=15), -2), (dict(ld_w=8), -2),
    (dict(ld_e=16 * 24 - 1), -2)])
def test_gated_refusals(pkg, bad, code):
    cfg = gated(pkg, **bad)
    assert pkg.moe_gated_forward_workspace_bytes(cfg) == 0 and pkg.moe_gated_backward_workspace_bytes(cfg) == 0
    assert pkg.moe_gated_forward(cfg, P, P, P, P, P, P, 0) == code
    assert pkg.moe_gated_backward(cfg, P, P, P, P, P, P, P, P, 0) == code


def test_gated_pointers(pkg):
    cfg = gated(pkg)
    assert 0 < pkg.moe_gated_forward_workspace_bytes(cfg) < pkg.moe_gated_backward_workspace_bytes(cfg)
    for i in range(6):
        a = [P] * 6
        a[i] = P + 1
        assert pkg.moe_gated_forward(cfg, *a, 0) == -3
        a[i] = None
        if i != 4:                                                              # gu may be left out
            assert pkg.moe_gated_forward(cfg, *a, 0) == -1
    assert pkg.moe_gated_forward(gated(pkg, grad_dtype=2, accumulate=1), *[P] * 6, 0) == -1
    ok = dict(dh=P, x=P, w=P, offsets=P, gu=P, dx=P, dw=P, ws=P)
    for name in ok:
        if name not in ("dx", "dw"):
            assert pkg.moe_gated_backward(cfg, *{**ok, name: None}.values(), 0) == -1, name
        assert pkg.moe_gated_backward(cfg, *{**ok, name: P + 1}.values(), 0) == -3, name
    assert pkg.moe_gated_backward(cfg, *{**ok, "dx": None, "dw": None}.values(), 0) == -1
    assert pkg.lib().moe_gated_forward(None, P, P, P, P, P, P, None) == -1


def vocab(pkg, **kw):
    a = dict(rows=4, V=10, d=16, dtype=0, grad_dtype=0, labels64=1, accumulate=0, copy_w=0, ld_x=0, ld_w=0, ld_dx=0)
    a.update(kw)
    return pkg.MoeVocabConfig(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(rows=-1), -1), (dict(V=0), -1), (dict(d=0), -1), (dict(dtype=2), -1), (dict(grad_dtype=1), -1),
    (dict(labels64=2), -1), (dict(accumulate=1), -1), (dict(accumulate=-1, grad_dtype=2), -1), (dict(copy_w=2), -1),
    (dict(rows=1 << 30), -2), (dict(V=1 << 30), -2), (dict(d=(1 << 20) + 1), -2), (dict(rows=1 << 29, V=1 << 29), -2),
    (dict(ld_x=15), -2), (dict(ld_w=8), -2), (dict(ld_dx=1 << 31), -2)])
def test_vocab_refusals(pkg, bad, code):
    cfg = vocab(pkg, **bad)
    assert pkg.moe_vocab_forward_workspace_bytes(cfg) == 0 and pkg.moe_vocab_backward_workspace_bytes(cfg) == 0
    assert pkg.moe_vocab_forward(cfg, *[P] * 6, 0) == code
    assert pkg.moe_vocab_backward(cfg, *[P] * 9, 0) == code


def test_vocab_pointers_and_workspace(pkg):
    cfg = vocab(pkg)
    for i in range(6):
        a = [P] * 6
        a[i] = None
        assert pkg.moe_vocab_forward(cfg, *a, 0) == -1
        a[i] = P + 1
        assert pkg.moe_vocab_forward(cfg, *a, 0) == -3
    names = ("dloss", "dlse", "x", "w", "labels", "lse", "dx", "dw", "ws")
    for name in names:
        a = dict.fromkeys(names, P)
        if name not in ("dloss", "dlse", "dx", "dw"):
            assert pkg.moe_vocab_backward(cfg, *{**a, name: None}.values(), 0) == -1, name
        assert pkg.moe_vocab_backward(cfg, *{**a, name: P + 1}.values(), 0) == -3, name
    a = dict.fromkeys(names, P)
    assert pkg.moe_vocab_backward(cfg, *{**a, "dloss": None, "dlse": None}.values(), 0) == -1
    assert pkg.moe_vocab_backward(cfg, *{**a, "dx": None, "dw": None}.values(), 0) == -1
    # w has to start its rows on 16-byte boundaries, or be copied
    assert pkg.moe_vocab_forward(cfg, P, P + 2, P, P, P, P, 0) == -3
    assert pkg.moe_vocab_forward(vocab(pkg, d=15), *[P] * 6, 0) == -3
    assert pkg.moe_vocab_forward_workspace_bytes(vocab(pkg, copy_w=1)) >= 10 * 16 * 2
    # a piece of the vocabulary, not all logits
    big = vocab(pkg, rows=16384, V=131072, d=4096)
    assert pkg.moe_vocab_backward_workspace_bytes(big) < 16384 * 131072 * 2 / 2
    assert pkg.moe_vocab_forward_workspace_bytes(big) < 16384 * 131072 * 2 / 8
    assert pkg.moe_vocab_backward_workspace_bytes(vocab(pkg, rows=0)) > 0


def grads(pkg, data, counts, types, outs=None, out_types=None, max_norm=1.0, eps=1e-6, norm=P, ws=P):
    d, c, t = array("Q", data), array("q", counts), array("i", types)
    at = lambda a: a.buffer_info()[0]  # noqa: E731
    if outs is None:
        return pkg.moe_grad_norm(at(d), at(c), at(t), len(d), norm, ws, 0)
    o, ot = array("Q", outs), array("i", out_types)
    return pkg.moe_grad_clip(pkg.MoeClipConfig(max_norm, eps), at(d), at(o), at(c), at(t), at(ot), len(d), norm, ws, 0)


def test_grad_refusals(pkg):
    assert pkg.moe_grad_workspace_bytes(-1) == 0 and pkg.moe_grad_workspace_bytes((1 << 24) + 1) == 0
    assert pkg.moe_grad_workspace_bytes(0) > 0 and pkg.moe_grad_workspace_bytes(5000) > pkg.moe_grad_workspace_bytes(5)
    assert pkg.moe_grad_norm(None, None, None, -1, P, P, 0) == -1
    assert pkg.moe_grad_norm(None, None, None, 2, P, P, 0) == -1
    for bad, code in [(dict(counts=[-1]), -1), (dict(types=[3]), -1), (dict(types=[-1]), -1), (dict(data=[0]), -1),
                      (dict(counts=[(1 << 42) + 1]), -2), (dict(data=[P + 1]), -3), (dict(types=[2], data=[P + 2]), -3),
                      (dict(norm=None), -1), (dict(ws=None), -1), (dict(norm=P + 1), -3), (dict(ws=P + 8), -3)]:
        a = dict(data=[P], counts=[4], types=[0])
        assert grads(pkg, **{**a, **bad}) == code, bad
        assert grads(pkg, **{**a, "outs": [P], "out_types": [0], **bad}) == (code if bad != dict(types=[2], data=[P + 2]) else -1)
    for bad in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=0.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(out_types=[1]), dict(outs=[0])):
        assert grads(pkg, **{**dict(data=[P], counts=[4], types=[0], outs=[P], out_types=[0]), **bad}) == -1, bad
    # outputs that share memory
    def clip(data, counts, outs, types=None, out_types=None):
        n = len(data)
        return grads(pkg, data, counts, types or [2] * n, outs, out_types or [2] * n)
    assert clip([P, P], [4, 4], [P, P]) == -1                                    # the same twice, in place
    assert clip([P, P + 12], [4, 4], [P, P + 12]) == -1                          # overlapping by one element
    assert clip([P], [4], [P + 4]) == -1                                         # shifted against itself
    assert clip([P, P + 16], [4, 4], [P + 16, P]) == -1                          # swapped
    assert clip([P, 2 * P], [4, 4], [3 * P, 3 * P + 8]) == -1                    # two outputs
    assert clip([P], [4], [P], types=[0], out_types=[2]) == -1                   # in place, but wider


def test_python_functions_check_before_they_call(pkg, monkeypatch):
    """Shapes, types and places are refused with a ValueError; CPU tensors too."""
    from mixture_experts_layer_device_gb300 import block
    monkeypatch.setattr(block, "_current_gpu", lambda: 0)
    x, w, off = torch.zeros(4, 8), torch.zeros(2, 6, 8), torch.zeros(3, dtype=torch.int32)
    for t in (x, x.bfloat16()):
        with pytest.raises(ValueError):
            block.gated_forward(t, w.to(t.dtype), off)
        with pytest.raises(ValueError):
            block.gated_backward(t, t, w.to(t.dtype), off, t)
        with pytest.raises(ValueError):
            block.vocab_loss_forward(t, t, off)
        with pytest.raises(ValueError):
            block.vocab_loss_backward(off, t, t, off, off)
        with pytest.raises(ValueError):
            block.grad_norm([t])
        with pytest.raises(ValueError):
            block.grad_clip([t], 1.0)


def test_config_layouts_match_the_header(pkg):
    assert ctypes.sizeof(pkg.MoeGatedConfig) == 8 + 7 * 4 + 4 + 5 * 8
    assert ctypes.sizeof(pkg.MoeVocabConfig) == 16 + 6 * 4 + 3 * 8
    assert ctypes.sizeof(pkg.MoeClipConfig) == 2 * 8


def test_clip_without_a_config(pkg):
    assert pkg.lib().moe_grad_clip(None, None, None, None, None, None, 0, P, P, None) == -1
