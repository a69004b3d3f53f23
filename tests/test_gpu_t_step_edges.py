"""The operators that end a training step where their values leave the ordinary
range, against the definitions (exact values where the inputs make them so)."""
import math

import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu

BF, HF, FP, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def blk():
    from mixture_experts_layer_device_gb300 import block
    return block


# ---------------------------------------------------------------- loss over a vocabulary
@pytest.mark.parametrize("V", [1, 700])
@pytest.mark.parametrize("rows", [3, 2100])      # the rows kernel within the gather, and before it
def test_vocab_infinite_logits(blk, V, rows):
    """lse as torch.logsumexp has it, loss = lse - z: NaN where the label's logit is infinite."""
    x = torch.zeros((rows, 64), dtype=BF, device="cuda")
    x[0, 0], x[1, 0] = 3e38, -3e38               # logits +inf and -inf where w is large
    w = torch.zeros((V, 64), dtype=BF, device="cuda")
    at = V - 1
    w[at, 0] = 3e38
    z = torch.zeros((3, V), dtype=F64)           # rows from 2 on are all like row 2
    z[0, at], z[1, at] = math.inf, -math.inf
    for label in {at, 0}:
        labels = torch.full((rows,), label, device="cuda")
        loss, lse = blk.vocab_loss_forward(x, w, labels)
        ref = torch.logsumexp(z, 1)
        for got, want in ((lse, ref), (loss, ref - z[:, label])):
            want = want.to(torch.float32).cuda()
            assert torch.allclose(got[:3], want, rtol=1e-6, atol=1e-6, equal_nan=True), (label, got[:3], want)
            assert torch.equal(got[2:], got[2:3].expand(rows - 2))


@pytest.mark.parametrize("dtype", [BF])          # fp16 does not reach such logits
@pytest.mark.parametrize("sign", [1, -1])
def test_vocab_logits_near_the_largest_number(blk, dtype, sign):
    """Logits of 1.5 2^127, whose product with log2 e is no fp32 number.  lse and loss are exact
    there (a step of fp32 is 2^104), and so is dz: 1 at the largest, 0 elsewhere."""
    V, d, far = 700, 64, slice(256, 384)
    x, w = torch.zeros((3, d), dtype=dtype, device="cuda"), torch.zeros((V, d), dtype=dtype, device="cuda")
    x[0, 0], x[1, 0] = sign * 2.0 ** 64, -sign * 2.0 ** 64
    w[far, 0] = 1.5 * 2.0 ** 63
    w[:, 1] = 0.25
    z = (x.to(F64) @ w.to(F64).T)
    top = 1.5 * 2.0 ** 127
    up = 0 if sign > 0 else 1                    # the row whose large logits are positive
    for label in (0, 300):
        labels = torch.full((3,), label, device="cuda")
        loss, lse = blk.vocab_loss_forward(x, w, labels)
        ref = torch.logsumexp(z, 1)
        assert float(lse[up]) == top and (float(loss[up]) == top if label == 0 else 0.0 <= float(loss[up]) < 4.9)  # log 128
        assert abs(float(lse[1 - up]) - math.log(V - 128)) < 1e-5
        assert float(loss[1 - up]) == pytest.approx(top if label == 300 else math.log(V - 128), rel=1e-6)
        assert abs(float(loss[2]) - math.log(V)) < 1e-5 and torch.allclose(lse.to(F64), ref, rtol=1e-6)
        one = torch.ones(3, device="cuda")
        dx = blk.vocab_loss_backward(None, x, w, labels, lse, dlse=one)[0]
        assert float(dx[up, 0]) == 128 * 1.5 * 2.0 ** 63 and float(dx[up, 1]) == 32.0
        assert float(dx[1 - up, 0]) == 0.0 and abs(float(dx[1 - up, 1]) - 0.25) < 1e-2
        dx = blk.vocab_loss_backward(one, x, w, labels, lse)[0]
        assert float(dx[up, 0]) == float(torch.tensor((128 if label == 0 else 127) * 1.5 * 2.0 ** 63).to(dtype))


def grows_evenly(rows, chain):
    """How far an fp32 sum of `rows` positive terms of one size may be off, relative to the sum:
    chains of additions at 2^-22 of the sum so far (half of the whole on average; a tensor
    core's truncating adder: four times a rounding), joined in fp32."""
    return (min(rows, chain) / 2 + 32) * 2.0 ** -22 + (rows / chain / 2 + 1) * 2.0 ** -24


@pytest.mark.parametrize("d", [64, 33])          # dw by TMA and element by element
@pytest.mark.parametrize("rows", [2048, 2049, 5000, 1 << 20])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_vocab_wide_gradient_of_many_rows(blk, rows, d, dtype):
    """An fp32 dw of terms of one sign: its error does not grow with the rows.  w = 0 makes every
    probability 2^-8, exactly, and dw[v] = 2^-8 sum_t x_t for all v."""
    V = 256
    g = torch.Generator(device="cuda").manual_seed(rows + d)
    x = torch.rand((rows, d), generator=g, device="cuda").to(dtype)
    w, labels = torch.zeros((V, d), dtype=dtype, device="cuda"), torch.zeros(rows, dtype=torch.int64, device="cuda")
    labels[::3] = -1                             # a third does not count
    lse = blk.vocab_loss_forward(x, w, labels)[1]
    ref = x[labels >= 0].to(F64).sum(0) / V
    one, n = torch.ones(rows, device="cuda"), int((labels >= 0).sum())
    run = lambda **kw: blk.vocab_loss_backward(None, x, w, labels, lse, dlse=one, need_dx=False, **kw)[1]  # noqa: E731
    dw = run(dw_dtype=FP)
    # 2^-20: lse and the exponential
    assert float((dw.to(F64) / ref - 1).abs().max()) <= grows_evenly(n, 2048) + 2.0 ** -20
    assert torch.equal(dw, run(dw_dtype=FP))
    acc = torch.rand((V, d), generator=g, device="cuda") * ref.float()
    total = ref + acc.to(F64)
    run(dw=acc, accumulate=True)
    assert float((acc.to(F64) / total - 1).abs().max()) <= grows_evenly(n, 2048) + 2.0 ** -20


@pytest.mark.parametrize("m,K", [(64, 64), (16, 33), (9, 33)])     # by TMA, and element by element
@pytest.mark.parametrize("rows", [65537, 1 << 20])
def test_narrow_gradients_of_many_rows(blk, rows, m, K):
    """A dw of 16 bits over many rows of one sign: its sum is off by less than its rounding.
    Chains of 65536 steps, an instruction of 16 terms truncated by at most 2^-22 of the sum so
    far (half of the whole on average), joined in fp32: 5e-4, and half a step of fp16."""
    g = torch.Generator(device="cuda").manual_seed(rows + m)
    x = torch.rand((rows, K), generator=g, device="cuda").to(HF)
    gu, dh = torch.ones((rows, 2 * m), dtype=HF, device="cuda"), torch.full((rows, m), 2.0 ** -8, dtype=HF, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    ref = x.to(F64).sum(0) / 256
    tol = 65536 / 16 / 2 * 2.0 ** -22 + 16 * 2.0 ** -24 + 2.0 ** -11
    dw = blk.gated_backward(dh, x, torch.zeros((1, 2 * m, K), dtype=HF, device="cuda"), off, gu, act="relu", need_dx=False)[1]
    assert dw.dtype == HF and float((dw.to(F64) / ref - 1).abs().max()) <= tol
    w, labels = torch.zeros((256, K), dtype=HF, device="cuda"), torch.zeros(rows, dtype=torch.int64, device="cuda")
    lse = blk.vocab_loss_forward(x, w, labels)[1]
    dw = blk.vocab_loss_backward(None, x, w, labels, lse, dlse=torch.ones(rows, device="cuda"), need_dx=False)[1]
    assert dw.dtype == HF and float((dw.to(F64) / ref - 1).abs().max()) <= tol + 2.0 ** -20


@pytest.mark.parametrize("cols", [1104, 1101])   # by TMA and element by element
def test_wide_gradients_of_many_rows_and_tiles(blk, cols):
    """Several accumulators per tile, several tiles per CTA pair, experts of one chain and of more:
    tolerances of test_gpu_r_step.py."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)  # noqa: E731
    off, m = [0, 9000, 9000, 17192, 17200, 36000], 900
    rows, E = off[-1], len(off) - 1
    x, w, dh, gu = rand(rows, cols), torch.zeros((E, 2 * m, cols), dtype=BF, device="cuda"), rand(rows, m), rand(rows, 2 * m)
    dw = blk.gated_backward(dh, x, w, torch.tensor(off, dtype=torch.int32, device="cuda"), gu, act="relu", need_dx=False,
                            dw_dtype=FP)[1]
    value = torch.clamp(gu[:, :m].double(), min=0.0)
    terms = torch.cat([dh.double() * gu[:, m:].double() * (gu[:, :m] > 0), dh.double() * value], 1)
    dgu = terms.to(BF).double()                  # as the products take it
    for e in range(E):
        a, b = off[e], off[e + 1]
        ref, size = dgu[a:b].T @ x[a:b].double(), dgu[a:b].abs().T @ x[a:b].double().abs()
        # where a product of three lies on the border of two bf16 numbers its fp32 form may round to the other
        slack = (2.0 ** -8 * terms[a:b].abs() * ((terms[a:b].float().to(BF).double() - dgu[a:b]) != 0)).T @ x[a:b].double().abs()
        tol = (b - a + 32) * 2.0 ** -22 * size + slack + 2.0 ** -20 * size
        assert bool(((dw[e].double() - ref).abs() <= tol).all()), e
    offsets, w = torch.tensor(off, dtype=torch.int32, device="cuda"), rand(E, 2 * m, cols)
    dx, both = blk.gated_backward(dh, x, w, offsets, gu, act="relu", dw_dtype=FP)     # beside the data gradient
    assert torch.equal(both, dw) and torch.equal(dx, blk.gated_backward(dh, x, w, offsets, gu, act="relu", need_dw=False)[0])
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        again = blk.gated_backward(dh, x, w, offsets, gu, act="relu", dw_dtype=FP)
    for _ in range(2):
        again[1].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    V, rows = 5000, 7000
    x, w = rand(rows, cols), rand(V, cols) * cols ** -0.5
    labels = torch.randint(-1, V, (rows,), generator=g, device="cuda")
    lse = blk.vocab_loss_forward(x, w, labels)[1]
    dloss = torch.rand(rows, generator=g, device="cuda")
    dw = blk.vocab_loss_backward(dloss, x, w, labels, lse, need_dx=False, dw_dtype=FP)[1]
    r = step.vocab_backward(dloss, None, x, w, labels, lse, 2.0 ** -8, cols + 32)
    assert bool(((dw.double() - r["dw"]).abs() <= r["tol_dw"] + 2.0 ** -24 * r["dw"].abs() + 2.0 ** -25).all())


# ---------------------------------------------------------------- gradients
def test_clip_without_a_limit(blk):
    """max_norm = inf scales nothing, whatever the norm but NaN (the quotient inf / inf is one)."""
    for bad, norm in ((math.inf, math.inf), (-math.inf, math.inf), (3e38, None), (math.nan, math.nan)):
        grads = [torch.ones(1000, device="cuda"), torch.full((70,), 3.0, dtype=BF, device="cuda")]
        grads[0][77] = bad
        keep = [t.clone() for t in grads]
        for out in (None, [torch.empty_like(t, dtype=FP) for t in grads]):
            got = blk.grad_clip(grads, math.inf, out=out)
            if norm is not None:
                assert torch.allclose(got, torch.tensor(norm, device="cuda"), equal_nan=True)
            for t, k in zip(out or grads, keep):
                assert bool(torch.isnan(t).all()) if bad != bad else torch.equal(t, k.to(t.dtype))
    limited = torch.ones(10, device="cuda")
    limited[3] = math.inf
    blk.grad_clip([limited], 3e38)               # a limit, if a large one: c = 0
    assert float(limited[0]) == 0.0 and bool(torch.isnan(limited[3]))


# ---------------------------------------------------------------- gated products
@pytest.mark.parametrize("m,K", [(64, 64), (9, 33)])     # dw by TMA and element by element
@pytest.mark.parametrize("rows", [2049, 9000, 1 << 20])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gated_and_grouped_wide_gradients_of_many_rows(blk, rows, m, K, dtype):
    """An fp32 dw of terms of one sign: its error does not grow with an expert's rows.  dg = du =
    2^-8 exactly, so that dw[e] = 2^-8 sum x[r] for all its rows."""
    g = torch.Generator(device="cuda").manual_seed(rows + m)
    x = torch.rand((rows, K), generator=g, device="cuda").to(dtype)
    w, gu = torch.zeros((3, 2 * m, K), dtype=dtype, device="cuda"), torch.ones((rows, 2 * m), dtype=dtype, device="cuda")
    dh = torch.full((rows, m), 2.0 ** -8, dtype=dtype, device="cuda")
    dy = torch.full((rows, 2 * m), 2.0 ** -8, dtype=dtype, device="cuda")
    off = [0, 700, 700, rows]
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    ref = torch.stack([x[a:b].to(F64).sum(0) / 256 for a, b in zip(off, off[1:])])[:, None, :].expand(3, 2 * m, K)
    tol = grows_evenly(rows, 8192) * ref
    for back in (lambda **kw: blk.gated_backward(dh, x, w, offsets, gu, act="relu", need_dx=False, **kw)[1],
                 lambda **kw: blk.grouped_backward(dy, x, w, offsets, need_dx=False, **kw)[1]):
        dw = back(dw_dtype=FP)
        assert bool(((dw.to(F64) - ref).abs() <= tol).all()) and torch.all(dw[1] == 0)
        assert torch.equal(dw, back(dw_dtype=FP))
        before = torch.rand((3, 2 * m, K), generator=g, device="cuda")
        acc = before.clone()
        back(dw=acc, accumulate=True)
        assert bool(((acc.to(F64) - before.to(F64) - ref).abs() <= tol + 2.0 ** -22 * acc.abs()).all())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("m", [8, 9])            # rows in 16-byte pieces and element by element
def test_gated_slopes_far_out(blk, act, m):
    """Gates whose square leaves fp32: act(g) is g or 0, act'(g) 1 or 0.  Exact: w has one 1 per row."""
    big = torch.tensor([1e3, 1e10, 2e19, 1e30, 3e38], dtype=F64).to(BF)
    gates = torch.cat([big, -big]).cuda()
    rows, K = gates.numel(), 2 * m
    gu = torch.ones((rows, 2 * m), dtype=BF, device="cuda")
    gu[:, :m] = gates[:, None]
    dh = torch.full((rows, m), 0.5, dtype=BF, device="cuda")
    w, x = torch.eye(K, dtype=BF, device="cuda")[None].contiguous(), torch.ones((rows, K), dtype=BF, device="cuda")
    dx = blk.gated_backward(dh, x, w, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), gu, act=act, need_dw=False)[0]
    assert torch.all(dx[:5, :m] == 0.5) and torch.all(dx[5:, :m] == 0.0)
    assert torch.equal(dx[:5, m:], 0.5 * gu[:5, :m]) and torch.all(dx[5:, m:] == 0.0)
