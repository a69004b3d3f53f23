"""GPU parity of the operators that end a training step (loss over a vocabulary,
gated products, norm and clipping of gradients) against the float64 oracle
(oracle/step.py), at the sizes and masks where they can go wrong.

Tolerances, element by element.  Products: (n + 32) 2^-22 S as for the grouped
products (n terms of absolute sum S: fp32 sums, a factor of four for a tensor
core's truncating adder), plus the output's rounding u |ref|.
  lse   the logits' error, the sum's: at most 600 additions in a row and the
        exponentials' 2^-22 relative, their argument's error 2^-24 |max| log2 e
  dx,dw dz is off by the logits' error and 2^-20 of its exponential and by its own
        rounding u (oracle: tol_*)
  h     |act'| <= 1.2 and |act| <= |g| carry g's and u's errors over; 2^-20 for the
        activation itself
  norm  all terms positive: 64 fp32 additions in a row, halved by the root, and its
        rounding; the factor c takes its error over
"""
import math

import numpy as np
import pytest
import torch

from oracle import step

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
BF, HF, FP, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
TINY = 2.0 ** -25     # half of fp16's smallest step


@pytest.fixture(scope="module")
def blk():
    from mixture_experts_layer_device_gb300 import block
    return block


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def draw(shape, dtype, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def near(got, ref, tol):
    """|got - ref| <= tol + the rounding of the output, everywhere."""
    assert got.shape == ref.shape
    assert bool(torch.isfinite(got).all())
    off = (got.to(F64) - ref).abs()
    tol = tol + U[got.dtype] * ref.abs() + TINY
    bad = off > tol
    assert not bool(bad.any()), (int(bad.sum()), float((off / tol).max()), int((off / tol).argmax()))


# ---------------------------------------------------------------- loss over a vocabulary
VOCAB = [
    # rows, V, d
    (1, 1, 1), (1, 100, 16), (2, 300, 8), (3, 257, 33), (17, 128, 64), (64, 129, 72), (128, 256, 128), (129, 1000, 136),
    (255, 33, 200), (257, 5001, 64), (300, 2500, 321), (515, 513, 520), (1030, 777, 96), (2100, 300, 40), (5, 20000, 256),
    (700, 4099, 1000),
]


def vocab_case(rows, V, d, dtype, seed, ignored=0.25, label_dtype=torch.int64):
    g = gen(seed)
    w = draw((V, d), dtype, g, 2.0 * d ** -0.5)
    labels = torch.randint(0, V, (rows,), generator=g, device="cuda")
    x = draw((rows, d), dtype, g)
    out = torch.rand(rows, generator=g, device="cuda") < ignored
    if rows > 2:
        labels[out] = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, -100, V)[out]
        x[out] = float("nan")
    return x, w, labels.to(label_dtype)


def check_vocab_forward(loss, lse, x, w, labels):
    r = step.vocab_forward(x, w, labels)
    tol_z = (x.shape[1] + 32) * 2.0 ** -22 * r["z_size"]
    tol = tol_z + 2.0 ** -24 * (3 * (r["lse"].abs() + r["z_size"]) + 600 + 8)
    tol[~r["keep"]] = 0.0
    near(lse, r["lse"], tol)
    near(loss, r["loss"], 2 * tol + 2.0 ** -24 * r["lse"].abs())
    assert torch.all(loss[~r["keep"]] == 0) and torch.all(lse[~r["keep"]] == 0)


@pytest.mark.parametrize("rows,V,d", VOCAB)
@pytest.mark.parametrize("dtype,label_dtype", [(BF, torch.int64), (HF, torch.int32)])
def test_vocab_forward(blk, rows, V, d, dtype, label_dtype):
    x, w, labels = vocab_case(rows, V, d, dtype, rows + V, label_dtype=label_dtype)
    loss, lse, ws = blk.vocab_loss_forward(x, w, labels, return_workspace=True)
    assert blk.grouped_status(ws) == 0
    check_vocab_forward(loss, lse, x, w, labels)
    again = blk.vocab_loss_forward(x, w, labels)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])


def check_vocab_backward(dx, dw, dloss, dlse, x, w, labels, lse, before=None):
    r = step.vocab_backward(dloss, dlse, x, w, labels, lse, U[x.dtype], x.shape[1] + 32)
    if dx is not None:
        near(dx, r["dx"], r["tol_dx"])
    if dw is not None:
        near(dw, r["dw"] + (0 if before is None else before.to(F64)), r["tol_dw"])


@pytest.mark.parametrize("rows,V,d", VOCAB)
@pytest.mark.parametrize("dtype,grad_dtype,use", [(BF, BF, "both"), (HF, FP, "loss"), (BF, FP, "lse"), (HF, HF, "mean")])
def test_vocab_backward(blk, rows, V, d, dtype, grad_dtype, use):
    g = gen(rows * 3 + V)
    x, w, labels = vocab_case(rows, V, d, dtype, rows + 7 * V)
    lse = blk.vocab_loss_forward(x, w, labels)[1]
    dloss = None if use == "lse" else torch.randn(rows, generator=g, device="cuda")
    if use == "mean":
        dloss = torch.full((rows,), 512.0 / rows, device="cuda")
    dlse = torch.randn(rows, generator=g, device="cuda") * 0.1 if use in ("both", "lse") else None
    if rows > 4 and use != "mean":       # rows without a gradient: what x holds there does not count
        for t in (dloss, dlse):
            if t is not None:
                t[::5] = 0.0
        x[::5] = float("inf")
    dx, dw, ws = blk.vocab_loss_backward(dloss, x, w, labels, lse, dlse=dlse, dw_dtype=grad_dtype, return_workspace=True)
    assert blk.grouped_status(ws) == 0 and dx.dtype == dtype and dw.dtype == grad_dtype
    check_vocab_backward(dx, dw, dloss, dlse, x, w, labels, lse)
    again = blk.vocab_loss_backward(dloss, x, w, labels, lse, dlse=dlse, dw_dtype=grad_dtype)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    only = blk.vocab_loss_backward(dloss, x, w, labels, lse, dlse=dlse, dw_dtype=grad_dtype, need_dw=False)
    assert torch.equal(only[0], dx) and only[1] is None
    only = blk.vocab_loss_backward(dloss, x, w, labels, lse, dlse=dlse, dw_dtype=grad_dtype, need_dx=False)
    assert torch.equal(only[1], dw) and only[0] is None
    if grad_dtype == FP:                 # added to what is there
        before = draw((V, d), FP, g)
        acc = before.clone()
        blk.vocab_loss_backward(dloss, x, w, labels, lse, dlse=dlse, dw=acc, accumulate=True, need_dx=False)
        check_vocab_backward(None, acc, dloss, dlse, x, w, labels, lse, before)


def test_vocab_pieces_of_the_vocabulary(blk):
    """More rows than a piece of the whole vocabulary has room for: dx joins the pieces."""
    rows, V, d = 70000, 8500, 24
    x, w, labels = vocab_case(rows, V, d, BF, 3, ignored=0.02)
    loss, lse = blk.vocab_loss_forward(x, w, labels)
    dloss = torch.rand(rows, generator=gen(4), device="cuda") / rows
    dx, dw = blk.vocab_loss_backward(dloss, x, w, labels, lse)
    for part in torch.arange(rows, device="cuda").split(9000):
        check_vocab_forward(loss[part], lse[part], x[part], w, labels[part])
        check_vocab_backward(dx[part], None, dloss[part], None, x[part], w, labels[part], lse[part])
    total, tol = torch.zeros(V, d, dtype=F64, device="cuda"), torch.zeros(V, d, dtype=F64, device="cuda")
    for part in torch.arange(rows, device="cuda").split(9000):
        r = step.vocab_backward(dloss[part], None, x[part], w, labels[part], lse[part], U[BF], d + 32)
        total += r["dw"]
        tol += r["tol_dw"] * (rows + 32) / (9000 + 32)
    near(dw, total, tol)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_vocab_strides_and_alignment(blk, dtype):
    rows, V, d = 150, 700, 88
    g = gen(5)
    wide_x, wide_w = draw((rows, 3 * d + 5), dtype, g), draw((V, 2 * d + 8), dtype, g, 0.2)
    labels = torch.randint(0, V, (2 * rows,), generator=g, device="cuda")[::2]
    dloss = torch.randn(2 * rows, generator=g, device="cuda")[::2]
    for x, w in [(wide_x[:, 3:3 + d], wide_w[:, :d]), (wide_x[:, :d], wide_w[:, 8:8 + d]), (wide_x[:, :d], wide_w[:, 3:3 + d]),
                 (wide_x[:, :d].t().contiguous().t(), wide_w[:, :d].t().contiguous().t())]:
        loss, lse = blk.vocab_loss_forward(x, w, labels)
        check_vocab_forward(loss, lse, x, w, labels)
        out = torch.full((rows, d + 11), 7.0, dtype=dtype, device="cuda")
        dx, dw = blk.vocab_loss_backward(dloss, x, w, labels, lse, dx=out[:, 5:5 + d])
        check_vocab_backward(dx, dw, dloss, None, x, w, labels, lse)
        assert torch.all(out[:, :5] == 7) and torch.all(out[:, 5 + d:] == 7)


def test_vocab_nothing_counts(blk):
    for rows in (0, 1, 300):
        x = torch.full((rows, 64), float("nan"), dtype=BF, device="cuda")
        w = draw((500, 64), BF, gen(6))
        labels = torch.full((rows,), -1, device="cuda")
        loss, lse = blk.vocab_loss_forward(x, w, labels)
        assert loss.shape == (rows,) and torch.all(loss == 0) and torch.all(lse == 0)
        dx, dw = blk.vocab_loss_backward(torch.ones(rows, device="cuda"), x, w, labels, lse)
        assert torch.all(dx == 0) and torch.all(dw == 0)
        acc = torch.full((500, 64), 3.0, device="cuda")
        blk.vocab_loss_backward(torch.ones(rows, device="cuda"), x, w, labels, lse, dw=acc, accumulate=True)
        assert torch.all(acc == 3)


def test_vocab_values_at_the_edges(blk):
    """Logits far apart, infinite ones, a row that is not finite: its neighbours keep their values."""
    V, d = 700, 64
    x, w, labels = vocab_case(40, V, d, BF, 8, ignored=0.0)
    x[3] *= 60.0                      # sure of one entry: the others' exponentials vanish
    x[5] = 0.0                        # all logits equal
    check_vocab_forward(*blk.vocab_loss_forward(x, w, labels), x, w, labels)
    clean = blk.vocab_loss_forward(x, w, labels)
    dloss = torch.ones(40, device="cuda")
    dx = blk.vocab_loss_backward(dloss, x, w, labels, clean[1])[0]
    check_vocab_backward(dx, None, dloss, None, x, w, labels, clean[1])
    bad = x.clone()
    bad[7] = float("nan")
    loss, lse = blk.vocab_loss_forward(bad, w, labels)
    assert bool(torch.isnan(loss[7])) and bool(torch.isnan(lse[7]))
    others = torch.arange(40, device="cuda") != 7
    assert torch.equal(loss[others], clean[0][others])
    dx2 = blk.vocab_loss_backward(dloss, bad, w, labels, lse)[0]
    assert torch.equal(dx2[others], dx[others]) and bool(torch.isnan(dx2[7]).all())
    dloss[9] = float("inf")           # an infinite coefficient stays in its row
    dx3 = blk.vocab_loss_backward(dloss, x, w, labels, clean[1])[0]
    others = torch.arange(40, device="cuda") != 9
    assert torch.equal(dx3[others], dx[others]) and not bool(torch.isfinite(dx3[9]).any())
    # an infinite logit: its row's log-sum is infinite
    big = torch.zeros(2, d, dtype=BF, device="cuda")
    big[0, 0] = 3e38
    wb = torch.zeros(V, d, dtype=BF, device="cuda")
    wb[600, 0] = 3e38
    loss, lse = blk.vocab_loss_forward(big, wb, torch.zeros(2, dtype=torch.int64, device="cuda"))
    assert float(lse[0]) == math.inf and abs(float(lse[1]) - math.log(V)) < 1e-5


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** 60])
def test_vocab_gradients_of_any_size(blk, scale):
    """dz is rounded relative to the largest coefficient: tiny and huge gradients lose nothing."""
    x, w, labels = vocab_case(50, 300, 64, BF, 9)
    lse = blk.vocab_loss_forward(x, w, labels)[1]
    dloss = torch.rand(50, generator=gen(10), device="cuda") + 0.5
    one = blk.vocab_loss_backward(dloss, x, w, labels, lse)
    two = blk.vocab_loss_backward(dloss * scale, x, w, labels, lse)
    for a, b in zip(one, two):
        assert torch.equal((a.double() * scale), b.double())


def test_vocab_offsets_past_32_bits(blk):
    """w of more than 2^31 elements; labels and sums at its far end."""
    V, d, rows = 540000, 4096, 3
    w = torch.zeros((V, d), dtype=BF, device="cuda")
    x = draw((rows, d), BF, gen(11))
    tail = draw((64, d), BF, gen(12), d ** -0.5)
    w[-64:] = tail
    labels = torch.tensor([V - 1, V - 64, 0], device="cuda")
    loss, lse = blk.vocab_loss_forward(x, w, labels)
    z = torch.cat([x.to(F64) @ tail.to(F64).T, torch.zeros(rows, 1, dtype=F64, device="cuda")], 1)
    z[:, -1] += math.log(V - 64)
    ref = torch.logsumexp(z, 1)
    assert float((lse.to(F64) - ref).abs().max()) < 1e-4
    assert float((loss.to(F64) - (ref - torch.stack([z[0, 63], z[1, 0], z[2, -1] * 0]))).abs().max()) < 1e-4
    dx, dw = blk.vocab_loss_backward(torch.ones(rows, device="cuda"), x, w, labels, lse)
    ref = step.vocab_backward(torch.ones(rows, device="cuda"), None, x, tail, labels - (V - 64), lse, U[BF], d + 32)
    far = dw[-64:].to(F64)
    p0 = torch.exp(-lse[2].to(F64))
    assert float((far[1:63] - (ref["dw"][1:63] + torch.exp(z[2, 1:63] - lse[2].to(F64))[:, None] * x[2].to(F64))).abs().max()) < 1e-2
    assert float((dw[0].to(F64) - ((torch.exp(-lse[:2].to(F64))[:, None] * x[:2].to(F64)).sum(0) + (p0 - 1) * x[2].to(F64))).abs().max()) < 2e-2


# ---------------------------------------------------------------- gated products
GATED = [
    # rows, E, m, K, rows before / after that belong to no expert
    (1, 1, 8, 8, 0, 0), (1, 5, 16, 24, 0, 0), (3, 4, 1, 1, 0, 0), (7, 3, 33, 17, 2, 1), (64, 64, 128, 64, 0, 0),
    (129, 2, 256, 128, 0, 3), (257, 3, 264, 136, 1, 1), (300, 40, 65, 67, 0, 0), (777, 9, 144, 200, 0, 0),
    (1030, 6, 257, 251, 3, 4), (1500, 3, 500, 640, 0, 0), (2000, 130, 136, 328, 0, 0), (5, 300, 48, 512, 0, 0),
    (10, 16, 96, 4096, 1, 0), (4000, 5, 72, 80, 0, 5), (2600, 2000, 16, 64, 0, 0), (3000, 1, 1000, 320, 0, 2),
]


def offsets_of(rows, E, before, seed, skew=True):
    rng = np.random.default_rng(seed)
    counts = rng.multinomial(rows, rng.dirichlet(np.full(E, 0.5 if skew else 50.0)))
    return [before + int(v) for v in np.concatenate([[0], np.cumsum(counts)])]


def on_gpu(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def check_gated_forward(h, gu, x, w, off, act):
    m = w.shape[1] // 2
    r = step.gated_forward(x, w, off, act)
    tol = (x.shape[1] + 32) * 2.0 ** -22 * r["gu_size"]
    if gu is not None:
        near(gu, r["gu"], tol)
    g, u = r["gu"][:, :m], r["gu"][:, m:]
    tg, tu = tol[:, :m], tol[:, m:]
    near(h, r["h"], 1.2 * tg * (u.abs() + tu) + r["value"].abs() * tu + 2.0 ** -20 * r["h"].abs())


@pytest.mark.parametrize("rows,E,m,K,before,after", GATED)
@pytest.mark.parametrize("dtype,act", [(BF, "silu"), (HF, "gelu"), (BF, "gelu_tanh"), (HF, "relu")])
def test_gated(blk, rows, E, m, K, before, after, dtype, act):
    g = gen(rows + m)
    off = offsets_of(rows, E, before, rows)
    total = before + rows + after
    x, w = draw((total, K), dtype, g), draw((E, 2 * m, K), dtype, g, 1.5 * K ** -0.5)
    outside = torch.ones(total, dtype=torch.bool, device="cuda")
    outside[before:before + rows] = False
    x[outside] = float("nan")
    h, gu, ws = blk.gated_forward(x, w, on_gpu(off), act=act, return_workspace=True)
    assert blk.grouped_status(ws) == 0
    assert torch.all(h[outside] == 0) and torch.all(gu[outside] == 0)
    check_gated_forward(h, gu, x, w, off, act)
    alone, none = blk.gated_forward(x, w, on_gpu(off), act=act, need_gu=False)
    assert none is None and torch.equal(alone, h)

    dh = draw((total, m), dtype, g)
    dh[outside] = float("inf")
    gu[outside] = float("nan")
    for dw_dtype in (dtype, FP):
        dx, dw, ws = blk.gated_backward(dh, x, w, on_gpu(off), gu, act=act, dw_dtype=dw_dtype, return_workspace=True)
        assert blk.grouped_status(ws) == 0
        r = step.gated_backward(dh, x, w, off, gu, act, U[dtype])
        near(dx, r["dx"], r["tol_dx"])
        near(dw, r["dw"], r["tol_dw"])
        assert torch.all(dx[outside] == 0)
    before_dw = draw((E, 2 * m, K), FP, g)
    acc = before_dw.clone()
    only = blk.gated_backward(dh, x, w, on_gpu(off), gu, act=act, dw=acc, accumulate=True, need_dx=False)
    assert only[0] is None
    near(acc, r["dw"] + before_dw.to(F64), r["tol_dw"])
    only = blk.gated_backward(dh, x, w, on_gpu(off), gu, act=act, need_dw=False)
    assert only[1] is None and torch.equal(only[0], dx)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_gated_strides_and_alignment(blk, dtype):
    rows, E, m, K = 333, 4, 80, 120
    g = gen(21)
    off = offsets_of(rows, E, 0, 2)
    wide_x, wide_h = draw((rows, 2 * K + 3), dtype, g), draw((rows, 3 * m + 1), dtype, g)
    wide_w = draw((E, 2 * m + 3, K + 16), dtype, g, K ** -0.5)
    for cx, cw, ch in [(0, 0, 0), (8, 8, 8), (3, 0, 1), (0, 5, 0)]:
        x, w, dh = wide_x[:, cx:cx + K], wide_w[:, 1:1 + 2 * m, cw:cw + K], wide_h[:, ch:ch + m]
        out = torch.full((rows, m + 9), 7.0, dtype=dtype, device="cuda")
        guf = torch.full((rows, 2 * m + 16), 7.0, dtype=dtype, device="cuda")
        h, gu = blk.gated_forward(x, w, on_gpu(off), out=out[:, ch:ch + m], gu=guf[:, cw:cw + 2 * m])
        check_gated_forward(h, gu, x, w, off, "silu")
        assert int((out == 7).sum()) >= rows * 9 and int((guf == 7).sum()) >= rows * 16
        dx, dw = blk.gated_backward(dh, x, w, on_gpu(off), gu)
        r = step.gated_backward(dh, x, w, off, gu, "silu", U[dtype])
        near(dx, r["dx"], r["tol_dx"])
        near(dw, r["dw"], r["tol_dw"])


@pytest.mark.parametrize("m,K", [(128, 256), (24, 40), (33, 17)])
def test_gated_bad_offsets_are_reported(blk, m, K):
    x, w = draw((50, K), BF, gen(22)), draw((3, 2 * m, K), BF, gen(23))
    for off in ([0, 20, 10, 50], [-1, 5, 20, 50], [0, 5, 20, 51]):
        ws = blk.gated_forward(x, w, on_gpu(off), return_workspace=True)[2]
        assert blk.grouped_status(ws) == -7
        ws = blk.gated_backward(x[:, :m].contiguous() if K >= m else draw((50, m), BF, gen(24)), x, w, on_gpu(off),
                                draw((50, 2 * m), BF, gen(25)), return_workspace=True)[2]
        assert blk.grouped_status(ws) == -7


def test_gated_without_rows(blk):
    w, off = draw((3, 32, 48), BF, gen(26)), torch.zeros(4, dtype=torch.int32, device="cuda")
    for rows in (0, 9):
        x = torch.full((rows, 48), float("nan"), dtype=BF, device="cuda")
        h, gu = blk.gated_forward(x, w, off)
        assert h.shape == (rows, 16) and gu.shape == (rows, 32) and torch.all(h == 0) and torch.all(gu == 0)
        dx, dw = blk.gated_backward(h, x, w, off, gu)
        assert torch.all(dx == 0) and torch.all(dw == 0) and dw.shape == w.shape


def test_gated_activations_die_out_exactly(blk):
    """Where an activation vanishes its value keeps its relative precision; large gates are the identity."""
    for act in ("silu", "gelu", "gelu_tanh", "relu"):
        gates = torch.tensor([-80.0, -20.0, -9.0, -5.0, -3.0, -1.0, -0.0, 0.0, 1.0, 5.0, 20.0, 300.0], device="cuda").to(BF)
        n = gates.numel()
        x = torch.zeros((n, 16), dtype=BF, device="cuda")
        x[:, 0], x[:, 1] = gates, 1.0
        w = torch.zeros((1, 16, 16), dtype=BF, device="cuda")
        w[0, :8, 0], w[0, 8:, 1] = 1.0, 1.0
        h, gu = blk.gated_forward(x, w, on_gpu([0, n]), act=act)
        ref = step.act(act, gates.to(F64))[0]
        assert float((h[:, 0].to(F64) - ref).abs().sub(2.0 ** -8 * 1.01 * ref.abs()).max()) <= 1e-37


# ---------------------------------------------------------------- gradients
def flat_tensors(sizes, dtypes, g, std=1.0, shift=0):
    """Tensors cut from one buffer per type, starting `shift` elements in."""
    out = []
    flats = {dt: draw((sum(s for s, d in zip(sizes, dtypes) if d == dt) + shift,), dt, g, std) for dt in set(dtypes)}
    at = {dt: shift for dt in flats}
    for s, dt in zip(sizes, dtypes):
        out.append(flats[dt][at[dt]:at[dt] + s])
        at[dt] += s
    return out


SIZES = [[1], [0], [7], [1, 1, 1], [16384], [16385, 3], [100000, 0, 5], [1 << 20, 333333, 1, 2, 3],
         list(range(1, 200)), [17] * 1500, [5000001, 64]]
NORM_TOL = 2.0 ** -19 + 2.0 ** -24


@pytest.mark.parametrize("i", range(len(SIZES)))
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32", "mixed"])
def test_grad_norm_and_clip(blk, i, kind):
    g = gen(i)
    sizes = SIZES[i]
    types = [{"bf16": BF, "fp16": HF, "fp32": FP, "mixed": (BF, HF, FP)[k % 3]}[kind] for k in range(len(sizes))]
    grads = flat_tensors(sizes, types, g, 0.5, shift=i % 5)
    ref = step.grad_norm(grads)
    norm = blk.grad_norm(grads)
    assert norm.shape == () and norm.dtype == FP and abs(float(norm) - ref) <= NORM_TOL * ref + 1e-45
    assert torch.equal(norm, blk.grad_norm(grads))
    keep = [t.clone() for t in grads]
    for limit in (0.3 * ref + 1e-3, 2.0 * ref + 1.0, 0.0, math.inf):
        c = step.grad_factor(keep, limit, 1e-6)
        for where in ("apart", "masters", "here"):
            work = flat_tensors(sizes, types, g, 0.0, shift=i % 5)
            for t, k in zip(work, keep):
                t.copy_(k)
            out = None if where == "here" else flat_tensors(sizes, types if where == "apart" else [FP] * len(sizes), g, 1.0,
                                                            shift=(i + 1) % 4)
            got = blk.grad_clip(work, limit, out=out)
            assert torch.equal(got, norm)
            for t, k, o in zip(work, keep, out or work):
                if where != "here":
                    assert torch.equal(t, k)
                refs = k.to(F64) * c
                near(o, refs, refs.abs() * (NORM_TOL + 2.0 ** -23))
                if limit > ref:
                    assert torch.equal(o, k.to(o.dtype))


def test_grad_norm_neither_overflows_nor_vanishes(blk):
    for value, dt in [(3e38, BF), (1e-38, BF), (6e4, HF), (6e-8, HF), (1e30, FP), (1e-30, FP), (1e-43, FP), (2.0 ** -56, FP)]:
        t = torch.full((100003,), value, dtype=dt, device="cuda")
        ref = float(t[0].double()) * math.sqrt(100003)
        norm = float(blk.grad_norm([t]))
        assert norm == math.inf if ref > 3.4028235e38 else abs(norm - ref) <= 1e-5 * ref + 1e-44, (value, norm, ref)
        out = torch.empty_like(t)
        blk.grad_clip([t], ref / 4, out=[out], eps=1e-45)
        if float(t[0]) / 4 >= torch.finfo(dt).tiny:      # below the normal range a quarter may round to nothing
            assert abs(float(out[77]) / float(t[77]) - 0.25) < 2.0 ** -8
    huge, small = torch.full((9,), 1e25, device="cuda"), torch.full((9,), 1e-25, device="cuda")
    assert abs(float(blk.grad_norm([huge, small])) / 3e25 - 1) < 1e-6
    zero = torch.zeros(1 << 20, device="cuda")
    assert float(blk.grad_norm([zero, small])) == pytest.approx(3e-25, rel=1e-6)
    assert float(blk.grad_norm([zero])) == 0.0 and float(blk.grad_norm([])) == 0.0
    blk.grad_clip([zero], 0.0)
    assert torch.all(zero == 0)


def test_grad_values_that_are_not_finite(blk):
    a, b = torch.ones(1000, device="cuda"), torch.ones(1000, device="cuda", dtype=BF)
    a[77] = math.inf
    assert float(blk.grad_norm([a, b])) == math.inf
    blk.grad_clip([a, b], 1.0)              # c = 0: as the formula says
    assert bool(torch.isnan(a[77])) and float(a[0]) == 0.0 and torch.all(b == 0)
    b[5] = math.nan
    assert math.isnan(float(blk.grad_norm([b])))
    blk.grad_clip([b], 1.0)
    assert bool(torch.isnan(b).all())


def test_grad_layouts(blk):
    """Any order of dimensions that fills its memory, unaligned starts, neighbours in one 16-byte unit."""
    g = gen(31)
    base = draw((64, 33, 5), BF, g)
    views = [base.permute(2, 0, 1)]
    flat = draw((1000,), BF, g)
    keep = flat.clone()
    assert abs(float(blk.grad_norm(views)) - step.grad_norm([base])) <= 1e-5 * step.grad_norm([base])
    blk.grad_clip([flat[3:5], flat[5:6], flat[6:501]], 0.25, eps=1e-6)
    c = step.grad_factor([keep[3:501]], 0.25, 1e-6)
    assert torch.equal(flat[:3], keep[:3]) and torch.equal(flat[501:], keep[501:])
    near(flat[3:501], keep[3:501].to(F64) * c, keep[3:501].to(F64).abs() * c * 2.0 ** -18)
    out = torch.empty((5, 64, 33), device="cuda")
    with pytest.raises(ValueError):         # another layout than the gradient's
        blk.grad_clip(views, 1.0, out=[out])
    master = torch.empty_like(views[0], dtype=FP)
    blk.grad_clip(views, math.inf, out=[master])
    assert torch.equal(master, views[0].float())


def test_grad_overlaps_are_refused(blk):
    t = draw((4000,), FP, gen(32))
    keep = t.clone()
    other = torch.empty_like(t)
    for grads, out in [([t, t], None), ([t[:100], t[99:200]], None), ([t[:100]], [t[1:101]]), ([t, keep], [other, other]),
                       ([t[:10], t[10:20]], [t[10:20], t[:10]])]:
        with pytest.raises(ValueError):
            blk.grad_clip(grads, 1.0, out=out)
    assert torch.equal(t, keep)
    blk.grad_clip([t[:100], t[:100]], 1.0, out=[other[:100], other[100:200]])      # read twice, written apart
    assert abs(float(blk.grad_norm([t, t])) - math.sqrt(2) * step.grad_norm([t])) < 1e-3


def test_grad_counts_past_32_bits(blk):
    n = (1 << 31) + 12345
    t = torch.zeros(n, dtype=BF, device="cuda")
    t[-1], t[0], t[1 << 31] = 3.0, 4.0, 12.0
    assert float(blk.grad_norm([t])) == 13.0
    blk.grad_clip([t], 6.5, eps=1e-9)
    assert float(t[-1]) == 1.5 and float(t[0]) == 2.0 and float(t[1 << 31]) == 6.0
