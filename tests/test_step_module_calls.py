"""CPU-only checks of how the calls that end a training step meet autograd: tensors
changed in place, the grad mode, refused calls.  CPU tensors pose as GPU tensors
and a stand-in for the library records its calls (as in test_block_calls.py)."""
import pytest
import torch

from mixture_experts_layer_device_gb300 import block, module
from test_block_calls import SIDE, Gpu, gpu, on  # noqa: F401
from test_step_calls import FP, gpu_step  # noqa: F401


# ---------------------------------------------------------------- changed in place
@pytest.mark.parametrize("given", [None, SIDE], ids=["current", "stream"])
def test_autograd_learns_of_clipped_tensors(gpu_step, given):  # noqa: F811
    """As torch's own operations in place: what a graph has saved of such a tensor is stale."""
    grads, out = [on(Gpu, 5, 3), on(Gpu, 4, dtype=FP)], [on(Gpu, 5, 3, dtype=FP), on(Gpu, 4, dtype=FP)]
    before = [t._version for t in grads + out]
    block.grad_norm(grads, stream=given)
    assert [t._version for t in grads + out] == before
    block.grad_clip(iter(grads), 1.0, out=iter(out), stream=given)
    assert [t._version for t in grads] == before[:2]
    assert all(t._version > v for t, v in zip(out, before[2:]))
    after = [t._version for t in out]
    block.grad_clip(grads, 1.0, stream=given)
    assert all(t._version > v for t, v in zip(grads, before)) and [t._version for t in out] == after
    leaf = torch.ones(4, requires_grad=True)
    part = grads[1].as_subclass(torch.Tensor)
    stale = (leaf * part).sum()
    block.grad_clip(grads, 1.0, stream=given)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        stale.backward()


@pytest.mark.parametrize("given", [None, SIDE], ids=["current", "stream"])
def test_autograd_learns_of_what_is_added_to(gpu_step, given):  # noqa: F811
    R, E, m, K, V = 6, 3, 4, 8, 7
    x, w, off, dh, gu = on(Gpu, R, K), on(Gpu, E, 2 * m, K), on(Gpu, E + 1, dtype=torch.int32), on(Gpu, R, m), on(Gpu, R, 2 * m)
    table, ids, r = on(Gpu, V, K), on(Gpu, R, dtype=torch.int64), on(Gpu, R, dtype=FP)
    calls = [(lambda **kw: block.gated_backward(dh, x, w, off, gu, **kw), "dw", (E, 2 * m, K)),
             (lambda **kw: block.grouped_backward(gu, x, w, off, **kw), "dw", (E, 2 * m, K)),
             (lambda **kw: block.vocab_loss_backward(r, x, table, ids, r, **kw), "dw", (V, K)),
             (lambda **kw: block.embed_backward(ids, x, V, **kw), "dtable", (V, K))]
    for call, name, shape in calls:
        t = on(Gpu, *shape, dtype=FP)
        was = t._version
        call(**{name: t}, accumulate=True, stream=given)
        assert t._version > was, name


# ---------------------------------------------------------------- grad mode
def test_inference_leaves_gate_and_up_out(monkeypatch):
    """Without a graph nothing reads [g | u]: it is neither allocated nor written."""
    asked = []

    def forward(x, w, offsets, act, need_gu):
        asked.append(need_gu)
        gu = x @ w[0].T
        return gu[:, :2] * gu[:, 2:], gu if need_gu else None

    monkeypatch.setattr(block, "gated_forward", forward)
    layer = module.GatedLinear(1, 2, 3, act="relu", dtype=torch.float32, device="cpu")
    x, offsets = torch.randn(5, 3), torch.tensor([0, 5], dtype=torch.int32)
    trained = layer(x, offsets)
    assert asked == [True] and trained.requires_grad
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            h = layer(x, offsets)
        assert asked[-1] is False and torch.equal(h, trained) and not h.requires_grad
    layer.weight.requires_grad_(False)
    assert not layer(x, offsets).requires_grad and asked[-1] is False
    assert layer(x.requires_grad_(), offsets).requires_grad and asked[-1] is True


# ---------------------------------------------------------------- masters
def test_a_refused_clipping_leaves_the_masters_alone(monkeypatch):
    def refuse(grads, max_norm, out=None, eps=1e-6):
        raise ValueError("refused")

    ps = [torch.nn.Parameter(torch.zeros(n, 2)) for n in (3, 4, 5)]
    ps[0].grad, ps[2].grad = torch.ones(3, 2), torch.ones(2, 5).t()
    masters = [p.detach().clone().requires_grad_() for p in ps]
    masters[1].grad, masters[2].grad = torch.ones(4, 2), torch.ones(5, 2)
    was = [m.grad for m in masters]
    kept = [None if g is None else g.clone() for g in was]

    def unchanged():
        return all(m.grad is g and (g is None or torch.equal(g, k)) for m, g, k in zip(masters, was, kept))

    monkeypatch.setattr(block, "grad_clip", refuse)
    with pytest.raises(ValueError, match="refused"):
        module.clip_gradients(ps, 1.0, masters)
    assert unchanged()
    monkeypatch.setattr(block, "grad_clip", lambda *a, **kw: "n")
    for bad in (torch.zeros(2, 3), torch.zeros(3, 2, dtype=torch.bfloat16), torch.zeros(3, 2, device="meta")):
        with pytest.raises(ValueError, match="master 0"):
            module.clip_gradients(ps, 1.0, [bad] + masters[1:])
        assert unchanged() and bad.grad is None
    assert module.clip_gradients(ps, 1.0, masters) == "n"
    assert masters[1].grad is None and masters[2].grad.stride() == ps[2].grad.stride() and masters[0].grad.shape == (3, 2)
