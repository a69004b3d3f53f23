"""The loss over a vocabulary at the hidden widths it is meant for, on both sides of what
changes with the width: from 2049 columns on the logits come from several accumulators, the
epilogue's groups share a tile's columns and a row's chains are joined; rows of 2048 and more
are gathered by a whole block, in one launch with the rows that count (up to 2048 rows) or
behind it.

Entries of x and w are small whole numbers over a power of two: every logit is exact, in any
order of its sum, and so the tolerances hold nothing for the products of the forward:
  lse   as in test_gpu_r_step.py without the logits' error
  dx,dw the same oracle, with no error of the logits
Gradients against differences along the gradient's own signs, where the slope is the sum of
its absolute values."""
import pytest
import torch

from oracle import step
from test_gpu_r_step import BF, F64, FP, HF, U, blk, gen, near  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = [
    # rows, V, d
    (5, 700, 2040), (5, 700, 2048), (3, 131, 2056), (300, 777, 2049), (300, 777, 2176), (257, 1000, 4104), (129, 260, 4096),
    (130, 513, 7168), (40, 513, 7168), (1, 300, 6145), (2048, 300, 2080), (2049, 300, 2047), (2100, 300, 2080), (2300, 140, 4097),
]


def whole_case(rows, V, d, dtype, seed):
    """Logits of standard deviation about 3: 16ths, at most 24 bits long."""
    g = gen(seed)
    draw = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda")  # noqa: E731
    shift = 2.0 ** -round(0.5 * torch.log2(torch.tensor(4.0 * d / 81)).item())
    x, w = (draw(rows, d) * shift).to(dtype), draw(V, d).to(dtype)
    labels = torch.randint(0, V, (rows,), generator=g, device="cuda")
    if rows > 2:
        out = torch.rand(rows, generator=g, device="cuda") < 0.25
        labels[out] = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, -100, V)[out]
        x[out] = float("nan")
    return x, w, labels


@pytest.mark.parametrize("rows,V,d", WIDE)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_vocab_forward_of_wide_rows(blk, rows, V, d, dtype):  # noqa: F811
    x, w, labels = whole_case(rows, V, d, dtype, rows + V + d)
    loss, lse, ws = blk.vocab_loss_forward(x, w, labels, return_workspace=True)
    assert blk.grouped_status(ws) == 0
    r = step.vocab_forward(x, w, labels)
    keep = r["keep"]
    size = torch.zeros_like(r["lse"])
    size[keep] = (x[keep].to(F64) @ w.to(F64).T).abs().max(1).values
    # the largest logit's product with log2 e, the exponentials, 600 additions in a row
    tol = 2.0 ** -24 * (3 * (r["lse"].abs() + size) + 600 + 8)
    tol[~keep] = 0.0
    near(lse, r["lse"], tol)
    near(loss, r["loss"], 2 * tol + 2.0 ** -24 * r["lse"].abs())
    assert torch.all(loss[~keep] == 0) and torch.all(lse[~keep] == 0)
    again = blk.vocab_loss_forward(x, w, labels)
    assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("rows,V,d", WIDE)
@pytest.mark.parametrize("dtype,grad_dtype", [(BF, BF), (HF, FP)])
def test_vocab_backward_of_wide_rows(blk, rows, V, d, dtype, grad_dtype):  # noqa: F811
    x, w, labels = whole_case(rows, V, d, dtype, rows + 3 * V + d)
    g = gen(rows + d)
    lse = blk.vocab_loss_forward(x, w, labels)[1]
    dloss, dlse = (torch.randn(rows, generator=g, device="cuda") for _ in range(2))
    dx, dw, ws = blk.vocab_loss_backward(dloss, x, w, labels, lse, dlse=dlse, dw_dtype=grad_dtype, return_workspace=True)
    assert blk.grouped_status(ws) == 0
    r = step.vocab_backward(dloss, dlse, x, w, labels, lse, U[dtype], 0)
    near(dx, r["dx"], r["tol_dx"])
    near(dw, r["dw"], r["tol_dw"])
    again = blk.vocab_loss_backward(dloss, x, w, labels, lse, dlse=dlse, dw_dtype=grad_dtype)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("which", ["x", "w"])
@pytest.mark.parametrize("rows,V,d", [(60, 400, 64), (40, 300, 2304)])
def test_vocab_gradients_against_differences_along_them(blk, rows, V, d, which):  # noqa: F811
    """(f(t + v) - f(t - v)) / 2 of the summed loss against grad . v for v = sign of the oracle's
    gradient times a power of two, t + v and t - v exact in bf16.  A log-sum's third derivative
    along v is at most sqrt(3) / 18 of the cube of the range 2 u of the logits' changes; its
    sixth, the losses' rounding (1e-5 a row) and the gradient's own (2^-8 of sum |grad v|,
    twice for dz) bound the difference: under a tenth of the slope, so that a missing term
    shows."""
    g = gen(rows + d)
    small = 2.0 ** -6 if d <= 64 else 2.0 ** -9      # the entries' step, and v's
    x, w = ((torch.randint(-48, 49, (n, d), generator=g, device="cuda") * small).to(BF) for n in (rows, V))
    labels = torch.randint(0, V, (rows,), generator=g, device="cuda")
    one = torch.ones(rows, device="cuda")
    lse = blk.vocab_loss_forward(x, w, labels)[1]
    grad = blk.vocab_loss_backward(one, x, w, labels, lse)[0 if which == "x" else 1].double()
    t = x if which == "x" else w
    exact = step.vocab_backward(one, None, x, w, labels, lse, U[BF], 0)
    v = (torch.sign(exact["dx" if which == "x" else "dw"]) * small).to(BF)
    assert torch.equal((t + v) - v, t) and torch.equal((t - v) + v, t)
    f = [blk.vocab_loss_forward(*((t + s * v, w) if which == "x" else (x, t + s * v)), labels)[0].double().sum() for s in (1, -1)]
    change = v.double() @ w.double().T if which == "x" else x.double() @ v.double().T
    u = float(change.abs().max())
    slope, size = float((grad * v.double()).sum()), float((grad * v.double()).abs().sum())
    tol = rows * (2 * u) ** 3 * 3 ** 0.5 / 18 / 6 + rows * 1e-5 + 3 * 2.0 ** -8 * size
    assert tol < 0.1 * abs(slope)
    assert abs(float(f[0] - f[1]) / 2 - slope) <= tol
