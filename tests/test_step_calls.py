"""CPU-only checks of what block.py and module.py do around the calls that end a
training step: in which stream's order their copies, allocations and launches
stand, which GPUs their tensors are on, that second derivatives are refused.
CPU tensors pose as GPU tensors, and a stand-in for the library records its
calls (as in test_block_calls.py)."""
import pytest
import torch

from mixture_experts_layer_device_gb300 import block, module
from test_block_calls import BF, MAIN, SIDE, Gpu, OtherGpu, crooked, gpu, on, spread  # noqa: F401

FP = torch.float32


@pytest.fixture
def gpu_step(gpu, monkeypatch):  # noqa: F811
    """gpu, with the plans of the step's calls forgotten and the bulk reads of tensors as methods."""
    for name in ("get_device", "is_contiguous", "numel", "data_ptr"):
        monkeypatch.setattr(block, {"get_device": "_device_of", "data_ptr": "_address"}.get(name, "_" + name),
                            lambda t, name=name: getattr(t, name)())
    plans = (block._gated_plan, block._vocab_plan, block._grad_workspace)
    for p in plans:
        p.cache_clear()
    yield gpu
    for p in plans:
        p.cache_clear()


def calls(make, vec):
    """(operator, its tensors, its options)."""
    R, E, m, K, V = 6, 3, 4, 8, 7
    x, w, off, dh, gu = make(R, K), make(E, 2 * m, K), vec(E + 1, torch.int32), make(R, m), make(R, 2 * m)
    table, labels, r = make(V, K), vec(R, torch.int64), vec(R, FP)
    return [
        (block.gated_forward, dict(x=x, w=w, offsets=off), {}),
        (block.gated_backward, dict(dh=dh, x=x, w=w, offsets=off, gu=gu), {}),
        (block.vocab_loss_forward, dict(x=x, w=table, labels=labels), {}),
        (block.vocab_loss_backward, dict(dloss=r, x=x, w=table, labels=labels, lse=r, dlse=r), {}),
    ]


CALLS = ["gated_forward", "gated_backward", "vocab_loss_forward", "vocab_loss_backward"]
OUTPUTS = [dict(out=((6, 4), BF), gu=((6, 8), BF)), dict(dx=((6, 8), BF), dw=((3, 8, 8), BF)),
           dict(loss=((6,), FP), lse=((6,), FP)), dict(dx=((6, 8), BF), dw=((7, 8), BF))]


@pytest.mark.parametrize("i", range(4), ids=CALLS)
@pytest.mark.parametrize("given", [None, SIDE, 22], ids=["current", "stream", "handle"])
def test_copies_and_memory_belong_to_the_stream_of_the_launch(gpu_step, i, given):
    fn, tensors, opts = calls(lambda *s: crooked(Gpu, *s), lambda n, dt: spread(Gpu, n, dt))[i]
    out = fn(**tensors, **opts, stream=given)
    stream = MAIN if given is None else SIDE
    launches = [e for e in gpu_step.log if e[0] == "launch"]
    assert len(launches) == 1 and launches[0][2] == stream.cuda_stream
    made = [e for e in gpu_step.log if e[0] in ("copy", "new")]
    assert {e[0] for e in made} == {"copy", "new"} and all(e[1] is stream for e in made), made
    assert gpu_step.stream is MAIN
    if given is not None:
        kept = {e[1:] for e in gpu_step.log if e[0] == "kept"}
        for t in tensors.values():
            assert (SIDE, t.untyped_storage().data_ptr()) in kept
        for t in out:
            assert (MAIN, t.untyped_storage().data_ptr()) in kept


@pytest.mark.parametrize("i", range(4), ids=CALLS)
def test_tensors_on_another_gpu_are_refused(gpu_step, i):
    fn, tensors, opts = calls(lambda *s: on(Gpu, *s), lambda n, dt: on(Gpu, n, dtype=dt))[i]
    fn(**tensors, **opts)
    launched = len([e for e in gpu_step.log if e[0] == "launch"])
    for name, t in tensors.items():
        for other in (OtherGpu, torch.Tensor):
            with pytest.raises(ValueError):
                fn(**{**tensors, name: t.as_subclass(other)}, **opts)
    for name, (shape, dt) in OUTPUTS[i].items():
        fn(**tensors, **opts, **{name: on(Gpu, *shape, dtype=dt)})
        for bad in (on(OtherGpu, *shape, dtype=dt), on(Gpu, *shape, dtype=torch.float64), on(Gpu, *shape[:-1], shape[-1] + 1, dtype=dt)):
            with pytest.raises(ValueError):
                fn(**tensors, **opts, **{name: bad})
    assert len([e for e in gpu_step.log if e[0] == "launch"]) == launched + len(OUTPUTS[i])
    gpu_step.current = 1
    with pytest.raises(ValueError):
        fn(**tensors, **opts)


@pytest.mark.parametrize("given", [None, SIDE], ids=["current", "stream"])
def test_gradients_and_their_stream(gpu_step, given):
    grads, out = [on(Gpu, 5, 3), on(Gpu, 4, dtype=FP)], [on(Gpu, 5, 3, dtype=FP), on(Gpu, 4, dtype=FP)]
    block.grad_norm(grads, stream=given)
    block.grad_clip(grads, 1.0, out=out, stream=given)
    stream = MAIN if given is None else SIDE
    assert [e[2] for e in gpu_step.log if e[0] == "launch"] == [stream.cuda_stream] * 2
    assert all(e[1] is stream for e in gpu_step.log if e[0] == "new")
    if given is not None:
        kept = {e[1:] for e in gpu_step.log if e[0] == "kept"}
        for t in grads + out:
            assert (SIDE, t.untyped_storage().data_ptr()) in kept
    launched = len([e for e in gpu_step.log if e[0] == "launch"])
    wide = on(Gpu, 5, 6)
    for bad, other in [([on(OtherGpu, 5)], None), ([on(Gpu, 5).as_subclass(torch.Tensor)], None), ([wide[:, :3]], None),
                       ([on(Gpu, 5, dtype=torch.float64)], None), ([on(Gpu, 5)], [on(OtherGpu, 5)]), ([on(Gpu, 5)], []),
                       ([on(Gpu, 5)], [on(Gpu, 4)]), ([on(Gpu, 5)], [on(Gpu, 5, dtype=torch.float16)]),
                       ([on(Gpu, 5, 3)], [on(Gpu, 3, 5).t()])]:
        with pytest.raises(ValueError):
            block.grad_clip(bad, 1.0, out=other)
        if other is None:
            with pytest.raises(ValueError):
                block.grad_norm(bad)
    for number in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=1.0, eps=0.0), dict(max_norm=1.0, eps=float("inf"))):
        with pytest.raises(ValueError):
            block.grad_clip(grads, **number)
    assert len([e for e in gpu_step.log if e[0] == "launch"]) == launched


def test_refused_options(gpu_step):
    (gf, g, _), (gb, h, _), (vf, v, _), (vb, b, _) = calls(lambda *s: on(Gpu, *s), lambda n, dt: on(Gpu, n, dtype=dt))
    odd = on(Gpu, 3, 7, 8)
    for fn, a in [(gf, dict(g, act="swish")), (gf, dict(g, w=odd)), (gf, dict(g, need_gu=False, gu=on(Gpu, 6, 8))),
                  (gb, dict(h, act="tanh")), (gb, dict(h, need_dx=False, need_dw=False)), (gb, dict(h, accumulate=True)),
                  (gb, dict(h, dw_dtype=torch.float16)), (vf, dict(v, labels=on(Gpu, 5, dtype=torch.int64))),
                  (vf, dict(v, labels=on(Gpu, 6, dtype=FP))), (vf, dict(v, w=on(Gpu, 7, 9))), (vf, dict(v, x=on(Gpu, 6, 8, dtype=FP))),
                  (vb, dict(b, dloss=None, dlse=None)), (vb, dict(b, lse=None)), (vb, dict(b, accumulate=True)),
                  (vb, dict(b, need_dx=False, need_dw=False)), (vb, dict(b, dw_dtype=torch.float64)),
                  (vb, dict(b, dloss=on(Gpu, 5, dtype=FP))), (vb, dict(b, dlse=on(Gpu, 6)))]:
        with pytest.raises(ValueError):
            fn(**a)
    assert not [e for e in gpu_step.log if e[0] == "launch"]


# ---------------------------------------------------------------- autograd
@pytest.fixture
def plain(monkeypatch):
    b = module.block
    monkeypatch.setattr(b, "gated_forward", lambda x, w, offsets, act, need_gu: (
        (x @ w[0, :2].T) * (x @ w[0, 2:].T), x @ w[0].T))
    monkeypatch.setattr(b, "gated_backward", lambda dh, x, w, offsets, gu, act, need_dx, need_dw: tuple(
        t.detach() for t in (torch.cat([dh * gu[:, 2:], dh * gu[:, :2]], 1) @ w[0],
                             (torch.cat([dh * gu[:, 2:], dh * gu[:, :2]], 1).T @ x)[None])))
    monkeypatch.setattr(b, "vocab_loss_forward", lambda x, w, labels: (
        torch.logsumexp(x @ w.T, 1) - (x @ w.T)[torch.arange(len(labels)), labels], torch.logsumexp(x @ w.T, 1)))

    def vocab_backward(dloss, x, w, labels, lse, dlse, need_dx, need_dw):
        zero = torch.zeros(x.shape[0])
        a, c = zero if dloss is None else dloss, zero if dlse is None else dlse
        dz = (a + c)[:, None] * torch.exp(x @ w.T - lse[:, None])
        dz[torch.arange(len(labels)), labels] -= a
        return (dz @ w).detach(), (dz.T @ x).detach()
    monkeypatch.setattr(b, "vocab_loss_backward", vocab_backward)


def leaf(*shape):
    return torch.randn(*shape, requires_grad=True)


def gated():
    x, w = leaf(5, 3), leaf(1, 4, 3)
    plain_form = lambda: (x @ w[0, :2].T) * (x @ w[0, 2:].T)  # noqa: E731
    return (x, w), lambda: module.GatedFunction.apply(x, w, torch.tensor([0, 5]), "relu"), plain_form


def vocab(which):
    x, w, labels = leaf(5, 3), leaf(7, 3), torch.tensor([0, 6, 2, 2, 5])
    z = lambda: x @ w.T  # noqa: E731
    plain_form = (lambda: torch.nn.functional.cross_entropy(z(), labels, reduction="none")) if which == 0 else \
        (lambda: torch.logsumexp(z(), 1))
    return (x, w), lambda: module.VocabLossFunction.apply(x, w, labels)[which], plain_form


MAKERS = [gated, lambda: vocab(0), lambda: vocab(1)]


@pytest.mark.parametrize("make", MAKERS, ids=["gated", "loss", "lse"])
def test_first_derivatives_pass(plain, make):
    leaves, run, plain_form = make()
    want = torch.autograd.grad(plain_form().square().sum(), leaves)
    for graph in (False, True):
        got = torch.autograd.grad(run().square().sum(), leaves, create_graph=graph)
        assert all(torch.allclose(a, b, atol=1e-5) for a, b in zip(got, want))


@pytest.mark.parametrize("make", MAKERS, ids=["gated", "loss", "lse"])
@pytest.mark.parametrize("square", [True, False])
def test_a_second_derivative_is_refused(plain, make, square):
    leaves, run, _ = make()
    y = run()
    g, = torch.autograd.grad((y.square() if square else y).sum(), leaves[0], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        (y.sum() + g.square().sum()).backward()


def test_clip_gradients_takes_what_has_a_gradient(monkeypatch):
    seen = []
    monkeypatch.setattr(block, "grad_clip", lambda grads, max_norm, out=None, eps=1e-6: seen.append((grads, max_norm, out)) or "n")
    ps = [torch.nn.Parameter(torch.zeros(3, 2)), torch.nn.Parameter(torch.zeros(4)), torch.nn.Parameter(torch.zeros(2, 5))]
    ps[0].grad, ps[2].grad = torch.ones(3, 2), torch.ones(5, 2).t()
    assert module.clip_gradients(iter(ps), 2.0) == "n"
    assert [id(g) for g in seen[0][0]] == [id(ps[0].grad), id(ps[2].grad)] and seen[0][1:] == (2.0, None)
    masters = [p.detach().clone().requires_grad_() for p in ps]
    masters[1].grad = torch.ones(4)
    kept = masters[0].grad = torch.empty(3, 2)
    module.clip_gradients(ps, 2.0, masters)
    out = seen[1][2]
    assert out[0] is kept and masters[0].grad is kept and masters[1].grad is None and out[1] is masters[2].grad
    assert out[1].stride() == ps[2].grad.stride() and out[1].dtype == torch.float32
    with pytest.raises(ValueError):
        module.clip_gradients(ps, 2.0, masters[:2])


def test_a_weight_of_another_shape_is_refused():
    with pytest.raises(ValueError):
        module.VocabLoss(7, 3, weight=torch.nn.Parameter(torch.zeros(7, 4)))
    w = torch.nn.Parameter(torch.zeros(7, 3))
    assert module.VocabLoss(7, 3, weight=w).weight is w
