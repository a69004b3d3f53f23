"""CPU-only checks of the autograd functions around the library's calls, with
plain arithmetic in the kernels' place: first derivatives pass, a second one is
refused instead of dropped."""
import pytest
import torch

from mixture_experts_layer_device_gb300 import module


@pytest.fixture
def plain(monkeypatch):
    """block.py's functions as plain operations on one expert and a post-norm-free block."""
    b = module.block
    monkeypatch.setattr(b, "grouped_forward", lambda x, w, offsets: x @ w[0].T)
    monkeypatch.setattr(b, "grouped_backward", lambda dy, x, w, offsets, need_dx, need_dw: (
        (dy @ w[0]).detach() if need_dx else None, (dy.T @ x)[None].detach() if need_dw else None))
    monkeypatch.setattr(b, "norm_forward", lambda x, f, gate, w_post, w_pre, **kw: (x + f, x + f, None, x[:, 0]))
    monkeypatch.setattr(b, "norm_backward", lambda dz, dh, *a, **kw: (
        sum(g for g in (dz, dh) if g is not None).detach().clone(),) * 2 + (None,) * 3)
    monkeypatch.setattr(b, "embed_forward", lambda ids, table, scale: scale * table[ids])
    monkeypatch.setattr(b, "embed_backward", lambda ids, dout, V, scale: torch.zeros(V, dout.shape[-1]).index_add_(
        0, ids, scale * dout.detach()))


class Layer:
    """y = x + W_gu's sum; every gradient a copy of dy or zeros."""
    def prepare_from(self, *w):
        self.w = [None if t is None else t.detach() for t in w]

    def new_saved(self):
        return object()

    def forward(self, x, logits, train, saved):
        return x.detach() + self.w[0].sum()

    def backward(self, dy, x, saved):
        gu, dn = (torch.zeros_like(t) for t in self.w[:2])
        return dict(dx=dy.detach().clone(), dlogits=torch.zeros(x.shape[0], 2), dW_gu=gu, dW_dn=dn, dWs_gu=None, dWs_dn=None)


def leaf(*shape):
    return torch.randn(*shape, requires_grad=True)


def grouped():
    x, w = leaf(5, 3), leaf(1, 4, 3)
    return (x, w), lambda: module.GroupedFunction.apply(x, w, torch.tensor([0, 5], dtype=torch.int32))


def norm():
    x, f = leaf(5, 3), leaf(5, 3)
    return (x, f), lambda: module.BlockNormFunction.apply(x, f, None, None, None, "none", False, True, 1.0, 1e-6)[1]


def moe():
    x, logits, gu, dn = leaf(5, 3), leaf(5, 2), leaf(2, 2, 3), leaf(2, 3, 1)
    layer = Layer()
    return (x, gu), lambda: module.MoEFunction.apply(x, logits, None, gu, dn, None, None, layer)


def embedding():
    table = leaf(7, 3)
    return (table,), lambda: module.EmbeddingFunction.apply(torch.tensor([0, 4, 4, 6]), table, 2.0)


@pytest.mark.parametrize("make", [grouped, norm, moe, embedding])
def test_first_derivatives_pass(plain, make):
    leaves, run = make()
    want = torch.autograd.grad(run().square().sum(), leaves)
    for g in want:
        assert not g.requires_grad
    got = torch.autograd.grad(run().square().sum(), leaves, create_graph=True)      # and may be asked for a graph
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("make", [grouped, norm, moe, embedding])
def test_a_second_derivative_is_refused(plain, make):
    """In a sum with a term of its own, where a dropped one would pass unseen."""
    leaves, run = make()
    y = run()
    g, = torch.autograd.grad(y.square().sum(), leaves[0], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        (y.sum() + g.square().sum()).backward()


@pytest.mark.parametrize("make", [grouped, norm, moe])
def test_a_second_derivative_through_what_was_saved_is_refused(plain, make):
    """The arriving gradient is a constant; the result still depends on the inputs."""
    leaves, run = make()
    y = run()
    g, = torch.autograd.grad(y.sum(), leaves[0], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        (y.sum() + g.square().sum()).backward()


def test_a_gradient_that_depends_on_nothing_stays_a_constant(plain):
    x, w = leaf(5, 3), torch.randn(1, 4, 3)
    y = module.GroupedFunction.apply(x, w, torch.tensor([0, 5], dtype=torch.int32))
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    assert not g.requires_grad
    (y.sum() + g.square().sum()).backward()
    assert torch.allclose(x.grad, g)


def test_the_backward_uses_the_forwards_numbers(plain, monkeypatch):
    """A scale or alpha given as a tensor that changes in place in between."""
    table, x, f, number = leaf(7, 3), leaf(5, 3), leaf(5, 3), torch.tensor(2.0)
    seen = []
    kept = module.block.norm_backward
    monkeypatch.setattr(module.block, "norm_backward", lambda *a, **kw: seen.append(float(kw["alpha"])) or kept(*a, **kw))
    y = module.EmbeddingFunction.apply(torch.tensor([0, 4]), table, number)
    z, h = module.BlockNormFunction.apply(x, f, None, None, None, "none", False, True, number, 1e-6)
    number.fill_(3.0)
    (y.sum() + h.sum()).backward()
    assert torch.equal(table.grad[4], torch.full((3,), 2.0)) and seen == [2.0]
