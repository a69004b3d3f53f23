"""The modules around the layer against torch in fp32 (autograd through plain
operations), and the example that trains with all of them.

Tolerance: the modules compute in bf16 storage with fp32 sums; a chain of a
forward and a backward rounds each tensor once (2^-9 relative on average), so
relative Frobenius errors stay within a few 2^-8; 2e-2 is used."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

TOL = 2e-2


def rel(a, b):
    return float((a.detach().float() - b.detach().float()).norm() / b.detach().float().norm())


def leaves(*ts):
    return [t.detach().float().requires_grad_() for t in ts]


def test_grouped_linear_trains_as_plain_matmuls():
    from mixture_experts_layer_device_gb300.module import GroupedLinear
    torch.manual_seed(0)
    off = [2, 40, 40, 131]
    m = GroupedLinear(3, 72, 136)
    x = torch.randn(140, 136, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    G = torch.randn(140, 72, device="cuda", dtype=torch.bfloat16)
    y = m(x, torch.tensor(off, dtype=torch.int32, device="cuda"))
    (y * G).sum().backward()
    xr, wr = leaves(x, m.weight)
    yr = torch.cat([xr[:2, :72] * 0] + [xr[off[e]:off[e + 1]] @ wr[e].T for e in range(3)] + [xr[131:, :72] * 0])
    (yr * G.float()).sum().backward()
    assert rel(y, yr) < TOL and rel(x.grad, xr.grad) < TOL and rel(m.weight.grad, wr.grad) < TOL
    assert torch.all(m.weight.grad[1] == 0) and torch.all(x.grad[:2] == 0) and torch.all(y[131:] == 0)
    m.weight.requires_grad_(False)          # a frozen weight: only dx
    x.grad = None
    (m(x, torch.tensor(off, dtype=torch.int32, device="cuda")) * G).sum().backward()
    assert rel(x.grad, xr.grad) < TOL


@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
@pytest.mark.parametrize("use", ["both", "z", "h"])
def test_block_norm_trains_as_plain_operations(gate, use):
    from mixture_experts_layer_device_gb300.module import BlockNorm
    torch.manual_seed(1)
    T, d = 50, 264
    bf = dict(device="cuda", dtype=torch.bfloat16)
    m = BlockNorm(d, gate=gate, alpha=0.5)
    with torch.no_grad():
        for p in m.parameters():
            p.add_(0.2 * torch.randn_like(p))
    x, f = torch.randn(T, d, requires_grad=True, **bf), torch.randn(T, d, requires_grad=True, **bf)
    g = {"row": (T,), "full": (T, d)}.get(gate)
    g = None if g is None else torch.randn(g, requires_grad=True, **bf)
    Gz, Gh = torch.randn(T, d, **bf), torch.randn(T, d, **bf)
    z, h = m(x, f, g)
    (((z * Gz).sum() if use != "h" else 0) + ((h * Gh).sum() if use != "z" else 0)).backward()
    xr, fr, wq, wp = leaves(x, f, m.w_post, m.w_pre)
    gr = leaves(m.w_gate if gate == "channel" else g)[0] if gate != "none" else torch.ones((), device="cuda")
    rms = lambda v: torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    zr = 0.5 * xr + (gr[:, None] if gate == "row" else gr) * (fr * rms(fr) * wq)
    hr = zr * rms(zr) * wp
    (((zr * Gz).sum() if use != "h" else 0) + ((hr * Gh).sum() if use != "z" else 0)).backward()
    assert rel(z, zr) < TOL and rel(h, hr) < TOL
    pairs = [(x, xr), (f, fr), (m.w_post, wq)] + ([(m.w_pre, wp)] if use != "z" else [])
    if gate != "none":
        pairs.append((m.w_gate if gate == "channel" else g, gr))
    for a, b in pairs:
        assert rel(a.grad, b.grad) < TOL
    if use == "z":
        assert m.w_pre.grad is None


def test_block_norm_without_a_block():
    from mixture_experts_layer_device_gb300.module import BlockNorm
    m = BlockNorm(64, post=False)
    x = torch.randn(5, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    z, h = m(x)
    assert torch.equal(z, x)
    xr, = leaves(x)
    (h.float().square() * torch.arange(64, device="cuda")).sum().backward()
    hr = xr * torch.rsqrt(xr.square().mean(1, keepdim=True) + 1e-6)
    (hr.square() * torch.arange(64, device="cuda")).sum().backward()
    assert rel(x.grad, xr.grad) < TOL
    with pytest.raises(ValueError):
        m(x, None, x)


def test_token_embedding_trains_as_indexing():
    from mixture_experts_layer_device_gb300.module import TokenEmbedding
    torch.manual_seed(2)
    m = TokenEmbedding(30, 48, scale=math.sqrt(48))
    ids = torch.randint(-1, 30, (4, 25), device="cuda")
    G = torch.randn(4, 25, 48, device="cuda", dtype=torch.bfloat16)
    y = m(ids)
    (y * G).sum().backward()
    wr, = leaves(m.weight)
    yr = torch.where((ids >= 0)[..., None], wr[ids.clamp(min=0)] * math.sqrt(48), 0.0)
    (yr * G.float()).sum().backward()
    assert y.shape == (4, 25, 48) and rel(y, yr) < TOL and rel(m.weight.grad, wr.grad) < TOL


def test_the_example_learns():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        import block_training
    finally:
        sys.path.pop(0)
    losses = block_training.train(steps=40, tokens=256, say=lambda s: None)
    assert abs(losses[0] - math.log(997)) < 2.0
    assert losses[-1] < 0.5 * losses[0], losses
