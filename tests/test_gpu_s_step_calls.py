"""GPU tests of the operators that end a training step as they are used: on other
streams, in captured graphs, two at once, as modules, together, and their
gradients against differences.

Tolerance of the module tests: as in test_gpu_p_block_modules.py (a chain of
bf16 roundings, a few 2^-8 in relative Frobenius norm): 2e-2."""
import os
import sys

import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu

BF, HF, FP, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
TOL = 2e-2


@pytest.fixture(scope="module")
def blk():
    from mixture_experts_layer_device_gb300 import block
    return block


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def draw(shape, dtype, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def turned(t):
    """The same values with the last two dimensions in the other order in memory."""
    return t.transpose(-1, -2).contiguous().transpose(-1, -2)


def rel(a, b):
    return float((a.detach().double() - b.detach().double()).norm() / b.detach().double().norm())


class Step:
    """Inputs of all the step's calls, and the calls."""

    def __init__(self, blk, seed=0, turn=False):
        self.blk, g = blk, gen(seed)
        R, E, m, K, V = 200, 3, 72, 136, 1500
        t = turned if turn else (lambda v: v)
        self.x, self.w, self.dh = t(draw((R, K), BF, g)), t(draw((E, 2 * m, K), BF, g, K ** -0.5)), t(draw((R, m), BF, g))
        self.off = torch.tensor([0, 30, 30, R], dtype=torch.int32, device="cuda")
        self.table, self.labels = t(draw((V, K), BF, g, K ** -0.5)), torch.randint(-1, V, (R,), generator=g, device="cuda")
        self.dloss = torch.rand(R, generator=g, device="cuda")
        self.grads = [draw((40, 50), BF, g), draw((77,), FP, g), draw((3, 5, 7), HF, g)]

    def run(self, stream=None):
        b = self.blk
        h, gu = b.gated_forward(self.x, self.w, self.off, act="gelu", stream=stream)
        out = [h, gu, *b.gated_backward(self.dh, self.x, self.w, self.off, gu, act="gelu", stream=stream)]
        loss, lse = b.vocab_loss_forward(self.x, self.table, self.labels, stream=stream)
        out += [loss, lse, *b.vocab_loss_backward(self.dloss, self.x, self.table, self.labels, lse, stream=stream)]
        with torch.cuda.stream(stream if not isinstance(stream, int) else torch.cuda.ExternalStream(stream)):
            masters = [torch.empty_like(t, dtype=FP) for t in self.grads]
        out += [b.grad_norm(self.grads, stream=stream), b.grad_clip(self.grads, 3.0, out=masters, stream=stream), *masters]
        return out


def test_a_call_on_another_stream_does_not_wait_for_the_current_one(blk):
    s = Step(blk, turn=True)
    want = s.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.run(side)                                 # its memory and kernels are there from here on
    torch.cuda.synchronize()
    busy, done = torch.cuda.Event(), torch.cuda.Event()
    torch.cuda._sleep(1_000_000_000)            # about half a second
    busy.record()
    got = s.run(side)
    done.record(side)
    done.synchronize()
    assert not busy.query()
    with torch.cuda.stream(side):
        same = [torch.equal(a, b) for a, b in zip(got, want)]
    assert len(got) == len(want) and all(same)
    by_handle = s.run(side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(by_handle, want))


def test_two_steps_at_once(blk):
    """On two streams at the same time, each with its own memory: the results of one after the other."""
    a, b = Step(blk, 1), Step(blk, 2)
    want = a.run(), b.run()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(a.run(s), b.run(t)) for _ in range(6)]
    torch.cuda.synchronize()
    for pair in got:
        for x, y in zip(pair, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_captured_and_replayed(blk):
    """Two graphs over one memory pool, replayed in turns with inputs that changed in place."""
    steps = [Step(blk, 3), Step(blk, 4)]
    pool, graphs, outs = None, [], []
    for s in steps:
        s.run()
    torch.cuda.synchronize()
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(s.run())
        pool = pool or g.pool()
        graphs.append(g)
    for seed in (5, 6):
        for s, g, out in zip(steps, graphs, outs):
            fresh = Step(blk, seed)
            for name in ("x", "w", "dh", "table", "labels", "dloss", "off"):
                getattr(s, name).copy_(getattr(fresh, name))
            s.off.copy_(torch.tensor([0, 10 * seed, 100, 190], dtype=torch.int32))
            for a, b in zip(s.grads, fresh.grads):
                a.copy_(b)
            s.labels[:seed * 10] = -1           # another number of rows that count
            g.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in out]
            assert all(torch.equal(p, q) for p, q in zip(got, s.run()))


@pytest.mark.parametrize("E", [1, 5, 416, 417, 500])
@pytest.mark.parametrize("rows", [66, 70, 75, 129, 200, 300])
def test_small_calls_with_their_rows_on_one_expert(blk, E, rows):
    """Tiles are smaller where all run in one round; with many experts another launch makes their table."""
    g = gen(E + rows)
    m, K = 40, 72
    x, w, dh = draw((rows, K), BF, g), draw((E, 2 * m, K), BF, g, K ** -0.5), draw((rows, 2 * m), BF, g)
    for e in {0, E // 2, E - 1}:
        off = [0] * (e + 1) + [rows] * (E - e)
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        y = blk.grouped_forward(x, w, offsets)
        h, gu = blk.gated_forward(x, w, offsets)
        dx = blk.grouped_backward(dh, x, w, offsets, need_dw=False)[0]
        ref = x.to(F64) @ w[e].to(F64).T
        size = x.to(F64).abs() @ w[e].to(F64).abs().T
        tol = 2.0 ** -8 * ref.abs() + (K + 32) * 2.0 ** -22 * size
        assert bool(((y.to(F64) - ref).abs() <= tol).all()) and torch.equal(y, gu)
        rh = torch.nn.functional.silu(ref[:, :m]) * ref[:, m:]
        assert bool(((h.to(F64) - rh).abs() <= 2.0 ** -8 * rh.abs() + 2.0 ** -12 * (1 + size[:, :m] * size[:, m:])).all())
        rx, sx = dh.to(F64) @ w[e].to(F64), dh.to(F64).abs() @ w[e].to(F64).abs()
        assert bool(((dx.to(F64) - rx).abs() <= 2.0 ** -8 * rx.abs() + (2 * m + 32) * 2.0 ** -22 * sx).all())


def test_calls_over_no_rows_have_a_status(blk):
    w, labels = draw((50, 64), BF, gen(50)), torch.empty(0, dtype=torch.int64, device="cuda")
    x, zero = torch.empty((0, 64), dtype=BF, device="cuda"), torch.empty(0, device="cuda")
    for _ in range(3):
        torch.full((1 << 16,), 0x7f, dtype=torch.uint8, device="cuda")      # memory that a workspace may get
        assert blk.grouped_status(blk.vocab_loss_forward(x, w, labels, return_workspace=True)[2]) == 0
        assert blk.grouped_status(blk.vocab_loss_backward(zero, x, w, labels, zero, return_workspace=True)[2]) == 0


def test_many_gradients_captured(blk):
    """Hundreds of tensors' addresses in a graph's launches."""
    g = gen(51)
    flat, out = draw((300000,), BF, g), torch.empty(300000, device="cuda")
    sizes = [200 + 3 * i for i in range(300)]
    grads, outs = list(flat[:sum(sizes)].split(sizes)), list(out[:sum(sizes)].split(sizes))
    want = blk.grad_clip(grads, 3.0, out=outs).clone(), out.clone()
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = blk.grad_clip(grads, 3.0, out=outs)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        n = sum(sizes)
        assert torch.equal(norm, want[0]) and torch.equal(out[:n], want[1][:n])
    flat.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) - float(want[0]) / 2) < 1e-5 * float(norm)


# ---------------------------------------------------------------- modules
def test_gated_linear_trains_as_plain_operations():
    from mixture_experts_layer_device_gb300.module import GatedLinear
    torch.manual_seed(0)
    off = [2, 40, 40, 131]
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        m = GatedLinear(3, 40, 136, act=act)
        x = torch.randn(140, 136, device="cuda", dtype=BF, requires_grad=True)
        G = torch.randn(140, 40, device="cuda", dtype=BF)
        offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        h = m(x, offsets)
        (h * G).sum().backward()
        xr, wr = x.detach().float().requires_grad_(), m.weight.detach().float().requires_grad_()
        f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "relu": torch.relu,
             "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[act]
        parts = [f(xr[off[e]:off[e + 1]] @ wr[e, :40].T) * (xr[off[e]:off[e + 1]] @ wr[e, 40:].T) for e in range(3)]
        hr = torch.cat([xr[:2, :40] * 0] + parts + [xr[131:, :40] * 0])
        (hr * G.float()).sum().backward()
        assert rel(h, hr) < TOL and rel(x.grad, xr.grad) < TOL and rel(m.weight.grad, wr.grad) < TOL
        assert torch.all(m.weight.grad[1] == 0) and torch.all(x.grad[:2] == 0) and torch.all(h[131:] == 0)
        with torch.no_grad():
            assert torch.equal(m(x, offsets), h)
        m.weight.requires_grad_(False)          # a frozen weight: only dx
        x.grad = None
        (m(x, offsets) * G).sum().backward()
        assert rel(x.grad, xr.grad) < TOL


@pytest.mark.parametrize("use", ["loss", "lse", "both"])
def test_vocab_loss_trains_as_cross_entropy(use):
    """With the embedding's own weight, which gets both gradients."""
    from mixture_experts_layer_device_gb300.module import TokenEmbedding, VocabLoss
    torch.manual_seed(1)
    V, d = 301, 72
    embed = TokenEmbedding(V, d)
    with torch.no_grad():
        embed.weight.mul_(8.0)
    head = VocabLoss(V, d, weight=embed.weight)
    ids, labels = torch.randint(0, V, (90,), device="cuda"), torch.randint(0, V, (90,), device="cuda")
    labels[::7] = -100
    loss, lse = head(embed(ids), labels)
    n = (labels >= 0).sum()
    pick = lambda a, b: {"loss": a, "lse": b, "both": a + b}[use]  # noqa: E731
    pick(loss.sum() / n, 1e-2 * lse.square().sum() / n).backward()
    wr = embed.weight.detach().float().requires_grad_()
    z = wr[ids].to(BF).float() @ wr.T
    z.retain_grad()
    keep = labels >= 0
    lr = torch.nn.functional.cross_entropy(z, labels, ignore_index=-100)
    sr = torch.logsumexp(z, 1)
    pick(lr, 1e-2 * sr[keep].square().sum() / n).backward()
    assert abs(float((loss.sum() / n).detach()) - float(lr.detach())) < 1e-4 and torch.allclose(lse[keep], sr[keep], atol=1e-4)
    assert torch.all(loss[~keep] == 0)
    assert rel(embed.weight.grad, wr.grad) < TOL


def test_clip_gradients_into_masters():
    from mixture_experts_layer_device_gb300.module import clip_gradients
    torch.manual_seed(2)
    ps = [torch.nn.Parameter(torch.randn(*s, device="cuda", dtype=BF)) for s in ((30, 40), (7,), (3, 4, 5))]
    for p in ps[:2]:
        p.grad = torch.randn_like(p)
    masters = [p.detach().float().requires_grad_() for p in ps]
    ref = step.grad_norm([p.grad for p in ps[:2]])
    c = step.grad_factor([p.grad for p in ps[:2]], 2.0, 1e-6)
    norm = clip_gradients(ps, 2.0, masters)
    assert abs(float(norm) - ref) < 1e-5 * ref and masters[2].grad is None
    for p, m in zip(ps[:2], masters):
        assert torch.allclose(m.grad.double(), p.grad.double() * c, rtol=1e-6, atol=0)
    at = masters[0].grad.data_ptr()
    clip_gradients(ps, 2.0, masters)
    assert masters[0].grad.data_ptr() == at
    clip_gradients(ps, 2.0)
    assert abs(step.grad_norm([p.grad for p in ps[:2]]) - 2.0) < 2e-2


# ---------------------------------------------------------------- together
def small_model(dtype=BF):
    """Embedding, norm, gated block, norm, loss: (parameters, loss function)."""
    from mixture_experts_layer_device_gb300.module import BlockNorm, GatedLinear, GroupedLinear, TokenEmbedding, VocabLoss
    torch.manual_seed(3)
    V, d, m, T = 501, 128, 96, 150
    embed, first = TokenEmbedding(V, d, scale=d ** 0.5), BlockNorm(d, post=False)
    up, down, last = GatedLinear(1, m, d), GroupedLinear(1, d, m), BlockNorm(d)
    head = VocabLoss(V, d)
    rows = torch.tensor([0, T], dtype=torch.int32, device="cuda")

    def loss(ids, labels):
        x, h = first(embed(ids))
        _, h = last(x, down(up(h, rows), rows))
        l, lse = head(h, labels)
        return (l.sum() + 1e-3 * lse.square().sum()) / (labels >= 0).sum()

    params = [p for mod in (embed, first, up, down, last, head) for p in mod.parameters()]

    def plain(ids, labels):
        ws = [p.detach().float().requires_grad_() for p in params]
        e, pre, wu, wd, post2, pre2, hw = ws
        rms = lambda v: torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
        x = e[ids] * d ** 0.5
        h = x * rms(x) * pre
        f = (torch.nn.functional.silu(h @ wu[0, :m].T) * (h @ wu[0, m:].T)) @ wd[0].T
        z = x + f * rms(f) * post2
        logits = (z * rms(z) * pre2) @ hw.T
        keep = labels >= 0
        l = torch.nn.functional.cross_entropy(logits[keep], labels[keep], reduction="sum")
        return (l + 1e-3 * torch.logsumexp(logits[keep], 1).square().sum()) / keep.sum(), ws

    ids, labels = (torch.randint(0, V, (T,), device="cuda") for _ in range(2))
    labels[5:20] = -1
    return params, loss, plain, ids, labels


def test_a_whole_step_together():
    """The operators as one training step against the same model in plain fp32 operations.
    Gradients pass some ten roundings to bf16: 5e-2 in relative norm."""
    from mixture_experts_layer_device_gb300.module import clip_gradients
    params, loss, plain, ids, labels = small_model()
    out = loss(ids, labels)
    out.backward()
    ref, ws = plain(ids, labels)
    ref.backward()
    assert abs(float(out) - float(ref)) < 2e-2 * float(ref)
    for p, w in zip(params, ws):
        assert rel(p.grad, w.grad) < 5e-2, tuple(p.shape)
    before = [p.grad.clone() for p in params]
    masters = [p.detach().float().requires_grad_() for p in params]
    norm = clip_gradients(params, 0.1, masters)
    want = step.grad_norm(before)
    assert abs(float(norm) - want) < 1e-5 * want
    c = step.grad_factor(before, 0.1, 1e-6)
    assert all(torch.allclose(m.grad.double(), g.double() * c, rtol=1e-6, atol=1e-30) for m, g in zip(masters, before))


def test_a_whole_step_captured():
    """Forward, backward and clipping of the modules in one graph, replayed on other tokens."""
    from mixture_experts_layer_device_gb300.module import clip_gradients
    params, loss, _, ids, labels = small_model()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):               # as captures of autograd want: warmed up on a side stream, nothing of it kept
        for _ in range(2):
            for p in params:
                p.grad = None
            loss(ids, labels).backward()
            clip_gradients(params, 0.1)
    torch.cuda.current_stream().wait_stream(side)
    for p in params:
        p.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = loss(ids, labels)
        out.backward()
        norm = clip_gradients(params, 0.1)
    ids.copy_(torch.randint(0, 501, ids.shape, device="cuda"))
    labels.copy_(torch.randint(-40, 501, ids.shape, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    got = [out.clone(), norm.clone()] + [p.grad.clone() for p in params]
    for p in params:
        p.grad = None
    with torch.cuda.stream(side):
        again = loss(ids, labels)
        again.backward()
        n = clip_gradients(params, 0.1)
    torch.cuda.synchronize()
    for a, b in zip(got, [again.detach(), n] + [p.grad for p in params]):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- differences
def test_vocab_gradients_against_differences(blk):
    """(f(x + v) - f(x - v)) / 2 of the summed loss against dx . v (and the same for w), with
    x + v and x - v exact in bf16.  A log-sum's third derivative along v is at most
    sqrt(3) / 18 of the cube of the range 2 u of the logits' changes; its sixth, the losses'
    rounding and dx's own (2^-8 of sum |dx v|, twice for dz) bound the difference."""
    rows, V, d = 60, 400, 64
    g = gen(40)
    x = (torch.randint(-48, 49, (rows, d), generator=g, device="cuda") / 64).to(BF)
    w = (torch.randint(-48, 49, (V, d), generator=g, device="cuda") / 64).to(BF)
    labels = torch.randint(0, V, (rows,), generator=g, device="cuda")
    one = torch.ones(rows, device="cuda")
    loss, lse = blk.vocab_loss_forward(x, w, labels)
    dx, dw = blk.vocab_loss_backward(one, x, w, labels, lse)
    for which, grad in (("x", dx), ("w", dw)):
        t = x if which == "x" else w
        v = ((torch.randint(0, 2, t.shape, generator=g, device="cuda") * 2 - 1) / 64).to(BF)
        f = [blk.vocab_loss_forward(*((t + s * v, w) if which == "x" else (x, t + s * v)), labels)[0].double().sum() for s in (1, -1)]
        assert torch.equal((t + v) - v, t) and torch.equal((t - v) + v, t)
        change = v.double() @ w.double().T if which == "x" else x.double() @ v.double().T
        u = float(change.abs().max())
        slope = float((grad.double() * v.double()).sum())
        tol = rows * (2 * u) ** 3 * 3 ** 0.5 / 18 / 6 + rows * 1e-5 + 3 * 2.0 ** -8 * float((grad.double() * v.double()).abs().sum())
        assert abs(float(f[0] - f[1]) / 2 - slope) <= tol and tol < 0.5 * abs(slope) + 3.0


def test_gated_gradients_against_differences(blk):
    """ReLU's gated product with gates that keep their sign is a polynomial of the second
    degree along any direction: differences are its slope.  Small whole numbers, exact in
    every step."""
    g = gen(41)
    R, m, K = 40, 16, 8
    x = torch.ones((R, K), device="cuda", dtype=BF)
    x[:, 1:] = torch.randint(-1, 2, (R, K - 1), generator=g, device="cuda").to(BF)
    w = torch.randint(-1, 2, (1, 2 * m, K), generator=g, device="cuda").to(BF)
    w[0, :m, 0] = 8                     # every gate is positive and stays so
    w[0, :m, 1:] *= (torch.arange(1, K, device="cuda") < 4).to(BF)
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    G = torch.randint(-2, 3, (R, m), generator=g, device="cuda").to(BF)
    h, gu = blk.gated_forward(x, w, off, act="relu")
    assert bool((gu[:, :m] > 4).all())
    dx, dw = blk.gated_backward(G, x, w, off, gu, act="relu", dw_dtype=FP)
    for which in ("x", "w"):
        t = x if which == "x" else w
        v = torch.randint(-1, 2, t.shape, generator=g, device="cuda").to(BF)
        if which == "x":
            v[:, 0] = 0
        else:
            v[:, :, 4:] = 0
            v[:, :m, 1:] = 0
        f = []
        for s in (1, -1):
            hs, gs = blk.gated_forward(*((t + s * v, w) if which == "x" else (x, t + s * v)), off, act="relu")
            assert bool((gs[:, :m] > 0).all()) and float(hs.abs().max()) <= 256
            f.append(float((hs.double() * G.double()).sum()))
        grad = dx if which == "x" else dw
        slope = float((grad.double() * v.double()).sum())
        # dx holds whole numbers up to 256 exactly; larger ones are rounded
        room = 0.0 if float(grad.abs().max()) <= 256 or which == "w" else 2.0 ** -8 * float((grad.double() * v.double()).abs().sum())
        assert abs((f[0] - f[1]) / 2 - slope) <= room


# ---------------------------------------------------------------- the example
def test_the_example_has_gradients_everywhere():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        import block_training
    finally:
        sys.path.pop(0)
    torch.manual_seed(4)
    model = block_training.Model(256)
    ids = torch.randint(0, 997, (256,), device="cuda")
    ids[::17] = -1
    model(ids).backward()
    for name, p in model.named_parameters():
        assert p.grad is not None and bool(torch.isfinite(p.grad).all()) and bool((p.grad != 0).any()), name
    used = torch.zeros(997, dtype=torch.bool, device="cuda")
    used[ids[ids >= 0]] = True
    assert torch.all(model.embed.weight.grad[~used] == 0)
