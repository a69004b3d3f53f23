"""Pins of the oracle of the operators around the layer against hand values and
central differences (CPU only)."""
import numpy as np
import pytest

from oracle import block as ob


def test_grouped_rows_use_their_expert_and_rows_of_no_expert_give_zero():
    W = np.stack([np.eye(2, 3), 10 * np.eye(2, 3)])
    x = np.arange(1.0, 16.0).reshape(5, 3)
    y, _ = ob.grouped_forward(x, W, [1, 3, 4])
    assert np.array_equal(y, [[0, 0], [4, 5], [7, 8], [100, 110], [0, 0]])


def test_grouped_backward_matches_differences():
    rng = np.random.default_rng(0)
    off = [1, 4, 4, 6]
    x, W, G = rng.standard_normal((7, 5)), rng.standard_normal((3, 4, 5)), rng.standard_normal((7, 4))
    dx, dW, _, _ = ob.grouped_backward(G, x, W, off)
    f = lambda a, b: float((G * ob.grouped_forward(a, b, off)[0]).sum())  # noqa: E731
    for _ in range(4):
        v, u = rng.standard_normal(x.shape), rng.standard_normal(W.shape)
        assert abs((f(x + v, W) - f(x - v, W)) / 2 - (dx * v).sum()) < 1e-10
        assert abs((f(x, W + u) - f(x, W - u)) / 2 - (dW * u).sum()) < 1e-10
    assert np.all(dW[1] == 0) and np.all(dx[0] == 0) and np.all(dx[6] == 0)


def test_norm_of_a_constant_row_and_residual():
    x, f = np.full((1, 4), 3.0), np.full((1, 4), -2.0)
    o = ob.norm_forward(x, f, None, None, None, alpha=2.0, eps=0.0)
    assert np.allclose(o["z"], 5.0) and np.allclose(o["h"], 1.0)
    assert np.allclose(o["r_post"], 0.5) and np.allclose(o["r_pre"], 0.2)


@pytest.mark.parametrize("kind", ["none", "channel", "row", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_norm_backward_matches_differences(kind, post, pre):
    rng = np.random.default_rng(3)
    T, d, eps, alpha = 3, 6, 1e-2, 0.7
    p = dict(x=rng.standard_normal((T, d)), f=rng.standard_normal((T, d)), wq=rng.standard_normal(d),
             wp=rng.standard_normal(d))
    shape = {"none": None, "channel": (d,), "row": (T,), "full": (T, d)}[kind]
    p["g"] = None if shape is None else rng.standard_normal(shape)
    Gz, Gh = rng.standard_normal((T, d)), rng.standard_normal((T, d))

    def fwd(q):
        return ob.norm_forward(q["x"], q["f"], q["g"], q["wq"], q["wp"], kind, post, pre, alpha, eps)

    def loss(q):
        o = fwd(q)
        return float((Gz * o["z"]).sum() + ((Gh * o["h"]).sum() if pre else 0.0))

    o = fwd(p)
    g, _ = ob.norm_backward(Gz, Gh if pre else None, o["z"], p["f"], p["g"], p["wq"], p["wp"], o["r_post"], o["r_pre"],
                            kind, post, pre, alpha)
    for name, grad in (("x", "dx"), ("f", "df"), ("g", "dgate"), ("wq", "dw_post"), ("wp", "dw_pre")):
        if g[grad] is None:
            continue
        v = rng.standard_normal(p[name].shape)
        h = 1e-5
        num = (loss({**p, name: p[name] + h * v}) - loss({**p, name: p[name] - h * v})) / (2 * h)
        assert abs(num - (g[grad] * v).sum()) < 1e-8, name


def test_embedding_padding_and_gradient():
    table = np.arange(6.0).reshape(3, 2)
    ids = [2, -1, 0, 2, 3]
    out = ob.embed_forward(ids, table, 2.0)
    assert np.array_equal(out, [[8, 10], [0, 0], [0, 2], [8, 10], [0, 0]])
    G = np.arange(10.0).reshape(5, 2)
    g, _ = ob.embed_backward(ids, G, 3, 2.0)
    assert np.array_equal(g, [[8, 10], [0, 0], [12, 16]])
    assert np.isclose((G * out).sum(), (g * table).sum())     # linear in the table
