"""The oracle of the operators that end a training step against differences and
torch's own derivatives in float64 (CPU)."""
import math

import pytest
import torch

from oracle import step

F = torch.float64


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F)


def differences(f, t, h=1e-5):
    """Central differences of the scalar f() in every element of t."""
    out = torch.zeros_like(t)
    for i in range(t.numel()):
        keep = float(t.view(-1)[i])
        t.view(-1)[i] = keep + h
        up = float(f())
        t.view(-1)[i] = keep - h
        out.view(-1)[i] = (up - float(f())) / (2 * h)
        t.view(-1)[i] = keep
    return out


def test_vocab_gradients_against_differences():
    x, w = rand(5, 3), rand(7, 3, seed=1)
    labels = torch.tensor([2, -1, 6, 7, 0])
    a, b = rand(5, seed=2), rand(5, seed=3)
    b[4], a[4] = 0.0, 0.0

    def f():
        r = step.vocab_forward(x, w, labels)
        return (a * r["loss"] + b * r["lse"]).sum()

    got = step.vocab_backward(a, b, x, w, labels, step.vocab_forward(x, w, labels)["lse"], 0.0, 0.0)
    assert torch.allclose(got["dx"], differences(f, x), atol=1e-8)
    assert torch.allclose(got["dw"], differences(f, w), atol=1e-8)
    assert torch.all(got["dx"][[1, 3, 4]] == 0)
    # torch's cross entropy is the same loss
    keep = torch.tensor([0, 2, 4])
    ce = torch.nn.functional.cross_entropy(x[keep] @ w.T, labels[keep], reduction="none")
    assert torch.allclose(ce, step.vocab_forward(x, w, labels)["loss"][keep])


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gated_gradients_against_differences(kind):
    x, w, off = rand(6, 4), rand(2, 6, 4, seed=1), [1, 3, 5]
    G = rand(6, 3, seed=2)
    fwd = step.gated_forward(x, w, off, kind)
    got = step.gated_backward(G, x, w, off, fwd["gu"], kind, 0.0)

    def f():
        return (G * step.gated_forward(x, w, off, kind)["h"]).sum()

    assert torch.allclose(got["dx"], differences(f, x), atol=1e-7)
    assert torch.allclose(got["dw"], differences(f, w), atol=1e-7)
    assert torch.all(got["dx"][[0, 5]] == 0)
    g = torch.linspace(-6, 6, 41, dtype=F, requires_grad=True)
    ref = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
           "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[kind](g)
    value, slope = step.act(kind, g.detach())
    slope_ref, = torch.autograd.grad(ref.sum(), g)
    assert torch.allclose(value, ref.detach(), atol=1e-12) and torch.allclose(slope, slope_ref, atol=1e-12)


def test_clipping_factor_is_torchs():
    grads = [rand(4, 3), rand(7, seed=1)]
    ps = [torch.nn.Parameter(torch.zeros_like(g)) for g in grads]
    for p, g in zip(ps, grads):
        p.grad = g.clone()
    total = torch.nn.utils.clip_grad_norm_(ps, 0.5)
    assert math.isclose(float(total), step.grad_norm(grads), rel_tol=1e-12)
    c = step.grad_factor(grads, 0.5, 1e-6)
    assert all(torch.allclose(p.grad, c * g, rtol=1e-12) for p, g in zip(ps, grads))
    assert step.grad_factor(grads, 100.0, 1e-6) == 1.0
