"""GPU parity of the operators around the layer (ragged grouped products, block
norms, token embedding) against the float64 oracle (oracle/block.py), at the
sizes and masks where they can go wrong.

Tolerance, element by element: u |ref| + (n + 32) 2^-22 S + tiny, with u the
unit roundoff of the output's type (bf16 2^-8, fp16 2^-11, fp32 2^-24; one
rounding per output), n the length of the longest fp32 sum behind the element
and S the oracle's sum of absolute values of its terms: n 2^-24 S bounds an
fp32 sum in any order, 2^-22 leaves a factor of four for a tensor core's
truncating adder and the few operations around the sum.  tiny is half of
fp16's smallest step."""
import numpy as np
import pytest
import torch

from oracle import block as ob

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def blk():
    from mixture_experts_layer_device_gb300 import block
    return block


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def draw(shape, dtype, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, ref, size, n):
    assert np.all(np.isfinite(f64(got)))
    tol = U[got.dtype] * np.abs(ref) + (n + 32) * 2.0 ** -22 * size + 2.0 ** -25
    err = np.abs(f64(got) - ref)
    worst = np.unravel_index(np.argmax(err / tol), err.shape) if err.size else None
    assert np.all(err <= tol), (worst, f64(got)[worst], ref[worst], tol[worst], int((err > tol).sum()))


def split(rows, E, how, seed):
    """Rows of every expert."""
    rng = np.random.default_rng(seed)
    if how == "one":
        c = np.zeros(E, dtype=np.int64)
        c[rng.integers(E)] = rows
        return c
    if how == "ends":            # only the first and the last expert
        c = np.zeros(E, dtype=np.int64)
        c[0], c[-1] = rows - rows // 3, rows // 3
        return c
    p = rng.dirichlet(np.full(E, 0.5 if how == "skew" else 50.0))
    return rng.multinomial(rows, p)


def offsets_of(counts, first=0):
    return torch.tensor(first + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


GROUPED = [
    # rows, E, N, K, split, rows before / after that belong to no expert
    (1, 1, 8, 8, "even", 0, 0),
    (1, 5, 16, 24, "one", 0, 0),
    (3, 4, 1, 1, "even", 0, 0),
    (7, 3, 33, 17, "skew", 2, 1),
    (64, 64, 128, 64, "even", 0, 0),
    (129, 2, 256, 128, "even", 0, 3),
    (255, 1, 264, 72, "one", 0, 0),
    (257, 3, 520, 136, "skew", 1, 1),
    (300, 40, 65, 67, "skew", 0, 0),
    (777, 9, 384, 200, "ends", 0, 0),
    (1030, 6, 513, 251, "skew", 3, 4),
    (1500, 3, 1000, 640, "even", 0, 0),
    (2000, 130, 264, 328, "skew", 0, 0),
    (5, 1024, 40, 512, "even", 0, 0),
    (3000, 1, 64, 64, "one", 1, 2),
    (2600, 2000, 16, 64, "skew", 0, 0),
    (4000, 5, 72, 80, "skew", 0, 5),
    (4000, 4, 301, 305, "skew", 2, 3),      # large and odd: padded copies
    (4000, 4, 304, 305, "ends", 0, 1),
    (4001, 5, 301, 304, "skew", 1, 0),
    (3, 300, 264, 256, "even", 0, 0),       # mostly experts without rows: their zeros written apart
    (3, 300, 263, 257, "even", 0, 0),
]


@pytest.mark.parametrize("rows,E,N,K,how,before,after", GROUPED)
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (HF, FP)])
def test_grouped_forward(blk, rows, E, N, K, how, before, after, dtype, out_dtype):
    g = gen(rows + N)
    counts = split(rows, E, how, rows)
    total = before + rows + after
    x, w = draw((total, K), dtype, g), draw((E, N, K), dtype, g, K ** -0.5)
    if before:
        x[:before] = float("nan")
    if after:
        x[-after:] = float("inf")
    off = offsets_of(counts, before)
    y = torch.full((total, N), 7.0, dtype=out_dtype, device="cuda")
    y2, ws = blk.grouped_forward(x, w, off, out=y, return_workspace=True)
    assert y2 is y and blk.grouped_status(ws) == 0
    xr = torch.nan_to_num(x, nan=0.0, posinf=0.0)
    ref, size = ob.grouped_forward(f64(xr), f64(w), off.cpu().numpy())
    close(y, ref, size, K)
    assert torch.equal(y, blk.grouped_forward(x, w, off, out_dtype=out_dtype))        # reproducible


@pytest.mark.parametrize("rows,E,N,K,how,before,after", GROUPED)
@pytest.mark.parametrize("dtype,dw_dtype", [(BF, BF), (HF, FP)])
def test_grouped_backward(blk, rows, E, N, K, how, before, after, dtype, dw_dtype):
    g = gen(rows + K)
    counts = split(rows, E, how, rows + 1)
    total = before + rows + after
    x, dy, w = draw((total, K), dtype, g), draw((total, N), dtype, g), draw((E, N, K), dtype, g, K ** -0.5)
    if before:
        x[:before], dy[:before] = float("nan"), float("inf")
    if after:
        x[-after:], dy[-after:] = float("-inf"), float("nan")
    off = offsets_of(counts, before)
    dx, dw, ws = blk.grouped_backward(dy, x, w, off, dw_dtype=dw_dtype, return_workspace=True)
    assert blk.grouped_status(ws) == 0
    xr, dyr = (torch.nan_to_num(t, nan=0.0, posinf=0.0, neginf=0.0) for t in (x, dy))
    rx, rw, sx, sw = ob.grouped_backward(f64(dyr), f64(xr), f64(w), off.cpu().numpy())
    close(dx, rx, sx, N)
    close(dw, rw, sw, int(counts.max()))
    dx2, dw2 = blk.grouped_backward(dy, x, w, off, dw_dtype=dw_dtype)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    only_dx, none = blk.grouped_backward(dy, x, w, off, need_dw=False)
    assert none is None and torch.equal(only_dx, dx)
    none, only_dw = blk.grouped_backward(dy, x, w, off, need_dx=False, dw_dtype=dw_dtype)
    assert none is None and torch.equal(only_dw, dw)


@pytest.mark.parametrize("N,K,pad", [(128, 192, 8), (72, 40, 1), (33, 65, 3)])
def test_grouped_accumulates_into_fp32_and_takes_strides(blk, N, K, pad):
    g = gen(5)
    E, rows = 5, 333
    counts = split(rows, E, "ends", 2)              # three experts get nothing
    off = offsets_of(counts)
    x = draw((rows, K + pad), BF, g)[:, :K]
    dy = draw((rows, N + 2 * pad), BF, g)[:, pad:pad + N]
    w = draw((E, N + 1, K + pad), BF, g, K ** -0.5)[:, 1:, :K]
    y = torch.zeros((rows, N + pad), dtype=BF, device="cuda")
    blk.grouped_forward(x, w, off, out=y[:, :N])
    ref, size = ob.grouped_forward(f64(x), f64(w), off.cpu().numpy())
    close(y[:, :N], ref, size, K)
    assert torch.all(y[:, N:] == 0)
    base = draw((E, N, K), FP, g)
    dw = base.clone()
    dx, dw2 = blk.grouped_backward(dy, x, w, off, dw=dw, accumulate=True)
    assert dw2 is dw
    rx, rw, sx, sw = ob.grouped_backward(f64(dy), f64(x), f64(w), off.cpu().numpy())
    close(dx, rx, sx, N)
    close(dw, f64(base) + rw, sw + np.abs(f64(base)), rows)
    for e in range(E):
        if counts[e] == 0:
            assert torch.equal(dw[e], base[e])


def test_grouped_zero_rows(blk):
    w = draw((3, 16, 24), BF, gen(0))
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = torch.empty((0, 24), dtype=BF, device="cuda"), torch.empty((0, 16), dtype=BF, device="cuda")
    assert blk.grouped_forward(x, w, off).shape == (0, 16)
    dx, dw = blk.grouped_backward(dy, x, w, off, dw=torch.full((3, 16, 24), 9.0, dtype=BF, device="cuda"))
    assert dx.shape == (0, 24) and torch.all(dw == 0)


@pytest.mark.parametrize("N,K", [(64, 64), (33, 65)])
@pytest.mark.parametrize("bad", [[0, 40, 20, 60], [0, -5, 20, 60], [0, 20, 40, 1 << 30], [-(1 << 31), 10, 20, 60]])
def test_grouped_bad_offsets_are_reported(blk, N, K, bad):
    g = gen(1)
    x, dy, w = draw((60, K), BF, g), draw((60, N), BF, g), draw((3, N, K), BF, g)
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    _, ws = blk.grouped_forward(x, w, off, return_workspace=True)
    assert blk.grouped_status(ws) == -7
    *_, ws = blk.grouped_backward(dy, x, w, off, return_workspace=True)
    assert blk.grouped_status(ws) == -7
    good = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device="cuda")
    y, ws = blk.grouped_forward(x, w, good, return_workspace=True)
    assert blk.grouped_status(ws) == 0
    close(y, *ob.grouped_forward(f64(x), f64(w), good.cpu().numpy()), K)


def test_grouped_gradient_against_differences(blk):
    """The products are linear in each argument: with fp32 outputs a central
    difference of <G, y> is <dx, v> and <dW, u> up to the roundings of y
    (2^-22 of the sums' sizes) and of dx (bf16)."""
    g = gen(9)
    rows, E, N, K = 200, 4, 48, 64
    off = offsets_of(split(rows, E, "skew", 0))
    q = lambda *s: (torch.randint(-8, 9, s, generator=g, device="cuda") / 8).to(BF)  # noqa: E731
    x, w, G, v, u = q(rows, K), q(E, N, K), q(rows, N), q(rows, K), q(E, N, K)
    dx, dw = blk.grouped_backward(G, x, w, off, dw_dtype=FP)
    f = lambda a, b: (G.double() * blk.grouped_forward(a, b, off, out_dtype=FP).double()).sum().item()  # noqa: E731
    slack = 2.0 ** -20 * rows * N * K
    num, want = (f(x + v, w) - f(x - v, w)) / 2, (dx.double() * v.double()).sum().item()
    assert abs(num - want) <= slack + 2.0 ** -8 * (dx.double().abs() * v.double().abs()).sum().item()
    num, want = (f(x, w + u) - f(x, w - u)) / 2, (dw.double() * u.double()).sum().item()
    assert abs(num - want) <= slack


def test_grouped_follows_the_routers_offsets(blk):
    """moe_route's offsets and perm drive the products directly."""
    import mixture_experts_layer_device_gb300 as pkg
    g = gen(4)
    T, E, k, d, n = 100, 12, 3, 64, 40
    cfg = pkg.config(T, 256, 128, E, k)
    logits = torch.randn((T, E), generator=g, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, cnt, off, perm = (torch.empty(s, **i32) for s in ((T, k), (E,), (E + 1,), (T * k,)))
    wts = torch.empty((T, k), dtype=FP, device="cuda")
    pkg.check(pkg.moe_route_noalloc(cfg, logits, idx, wts, cnt, off, perm))
    x, w = draw((T, d), BF, g), draw((E, n, d), BF, g, d ** -0.5)
    rows = torch.empty((T * k, d), dtype=BF, device="cuda")
    rows[perm.long()] = x.repeat_interleave(k, 0)
    y = blk.grouped_forward(rows, w, off)[perm.long()].view(T, k, n)
    ref = np.einsum("td,tknd->tkn", f64(x), f64(w)[idx.cpu().numpy()])
    size = np.einsum("td,tknd->tkn", np.abs(f64(x)), np.abs(f64(w)[idx.cpu().numpy()]))
    close(y, ref, size, d)


# ---------------------------------------------------------------- norms
NORM = [(1, 1), (1, 7168), (2, 8), (5, 33), (17, 512), (9, 520), (33, 1000), (3, 2883), (40, 4096), (2, 8200), (3, 16392),
        (700, 264), (400, 1024), (333, 4104), (160, 7168), (157, 8192), (170, 13000), (300, 2883), (200, 515), (161, 777),
        (1000, 40), (5000, 256)]


def norm_inputs(rows, d, dtype, kind, seed):
    g = gen(seed)
    x, f = draw((rows, d), dtype, g), draw((rows, d), dtype, g, 3.0)
    w_post, w_pre = (1 + draw((d,), FP, g, 0.3)).to(dtype), (1 + draw((d,), FP, g, 0.3)).to(dtype)
    shape = {"none": None, "channel": (d,), "row": (rows,), "full": (rows, d)}[kind]
    return x, f, None if shape is None else draw(shape, dtype, g), w_post, w_pre


def check_norm(blk, rows, d, dtype, kind, post, pre, alpha, weights=True, seed=0, eps=1e-5):
    x, f, gate, w_post, w_pre = norm_inputs(rows, d, dtype, kind, seed)
    if not weights:
        w_post = w_pre = None
    kw = dict(gate_kind=kind, post=post, pre=pre, alpha=alpha)
    z, h, r_post, r_pre = blk.norm_forward(x, f, gate, w_post, w_pre, eps=eps, **kw)
    o = ob.norm_forward(f64(x), f64(f), f64(gate), f64(w_post), f64(w_pre), kind, post, pre, alpha, eps)
    close(z, o["z"], o["z_size"], d)
    if post:
        close(r_post, o["r_post"], o["r_post"], d)
    if pre:
        # z's own error, of relative size (d + 32) 2^-22 of its terms, passes on to rms(z)
        amp = np.abs(o["z_size"]).max(1) / np.sqrt((o["z"] ** 2).mean(1))
        close(r_pre, o["r_pre"], o["r_pre"] * (1 + amp), d)
        close(h, o["h"], o["h_size"] * (2 + amp[:, None]), d)
    else:
        assert h is None and r_pre is None
    g = gen(seed + 1)
    dz, dh = draw((rows, d), dtype, g), draw((rows, d), dtype, g) if pre else None
    got = blk.norm_backward(dz, dh, z, f, gate, w_post, w_pre, r_post, r_pre, **kw)
    ref, size = ob.norm_backward(f64(dz), f64(dh), f64(z), f64(f), f64(gate), f64(w_post), f64(w_pre), f64(r_post),
                                 f64(r_pre), kind, post, pre, alpha)
    for name, t in zip(("dx", "df", "dgate", "dw_post", "dw_pre"), got):
        if name.startswith("dw") and not weights:
            assert t is None
            continue
        assert (t is None) == (ref[name] is None), name
        if t is not None:
            # the sums over a row feed every element of it: its rows' longest sums add up
            close(t, ref[name], size[name], d + (rows if t.dim() == 1 else 0))
    again = blk.norm_backward(dz, dh, z, f, gate, w_post, w_pre, r_post, r_pre, **kw)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("rows,d", NORM)
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_norm_sizes(blk, rows, d, dtype):
    check_norm(blk, rows, d, dtype, "channel", True, True, 0.5, seed=rows + d)


@pytest.mark.parametrize("kind", ["none", "channel", "row", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("rows,d", [(37, 264), (37, 1027), (5, 9000), (333, 1032), (311, 1027)])
def test_norm_gates_and_halves(blk, kind, post, pre, rows, d):
    check_norm(blk, rows, d, BF, kind, post, pre, 1.0, seed=7)


def test_norm_without_weights_and_plain_residual(blk):
    check_norm(blk, 20, 640, HF, "none", True, True, 1.0, weights=False)
    check_norm(blk, 20, 641, FP, "row", False, True, 0.25, weights=False)


def test_norm_pre_only_and_one_gradient(blk):
    g = gen(2)
    x, w = draw((9, 300), BF, g), draw((300,), BF, g)
    z, h, _, r = blk.norm_forward(x, None, None, None, w, need_z=False)
    assert z is None
    o = ob.norm_forward(f64(x), None, None, None, f64(w))
    close(h, o["h"], o["h_size"], 300)
    dh = draw((9, 300), BF, g)
    dx, df, dg, dwq, dw = blk.norm_backward(None, dh, x, None, None, None, w, None, r)
    ref, size = ob.norm_backward(None, f64(dh), f64(x), None, None, None, f64(w), None, f64(r))
    close(dx, ref["dx"], size["dx"], 300)
    close(dw, ref["dw_pre"], size["dw_pre"], 309)
    assert df is None and dg is None and dwq is None


def test_norm_strides_and_no_rows(blk):
    g = gen(6)
    rows, d = 11, 256
    wide = draw((rows, 3 * d), BF, g)
    x, f, gate = wide[:, :d], wide[:, d:2 * d], wide[:, 2 * d:]
    w = draw((d,), BF, g)
    zb = torch.zeros((rows, d + 3), dtype=BF, device="cuda")
    z, h, rq, rp = blk.norm_forward(x, f, gate, w, w, gate_kind="full", z=zb[:, :d])
    want = blk.norm_forward(x.contiguous(), f.contiguous(), gate.contiguous(), w, w, gate_kind="full")
    # an unaligned output takes another kernel: same numbers up to one rounding
    assert (z.float() - want[0].float()).abs().max() <= 2.0 ** -7 * want[0].float().abs().max()
    assert torch.all(zb[:, d:] == 0)
    got = blk.norm_backward(h, h, z, f, gate, w, w, rq, rp, gate_kind="full")
    ref, size = ob.norm_backward(*(f64(t) for t in (h, h, z, f, gate, w, w, rq, rp)), kind="full")
    for name, t in zip(("dx", "df", "dgate", "dw_post", "dw_pre"), got):
        close(t, ref[name], size[name], d + rows)
    e = torch.empty((0, d), dtype=BF, device="cuda")
    z, h, rq, rp = blk.norm_forward(e, e, None, w, w)
    assert z.shape == h.shape == (0, d)
    dx, df, _, dwq, dwp = blk.norm_backward(e, e, e, e, None, w, w, rq, rp)
    assert torch.all(dwq == 0) and torch.all(dwp == 0) and dx.shape == df.shape == (0, d)


def test_norm_zero_rows_and_infinities_stay_in_their_rows(blk):
    """rms(0) = sqrt(eps): zero rows give zeros; a row with NaN harms no other."""
    g = gen(8)
    x, f, w = draw((6, 128), BF, g), draw((6, 128), BF, g), draw((128,), BF, g)
    x[1] = f[1] = 0
    clean = blk.norm_forward(x, f, None, w, w)
    assert torch.all(clean[0][1] == 0) and torch.all(clean[1][1] == 0)
    f[3, 5] = float("nan")
    x[4, 7] = float("inf")
    z, h, rq, rp = blk.norm_forward(x, f, None, w, w)
    for r in (0, 1, 2, 5):
        assert torch.equal(z[r], clean[0][r]) and torch.equal(h[r], clean[1][r])
    assert torch.all(z[3].isnan()) and torch.all(h[3].isnan())


def test_norm_gradient_against_differences(blk):
    """fp32: central differences of <Gz, z> + <Gh, h> with a step of 2^-6 are off
    by h^2 / 6 of the third derivative (of order 1 here) times the number of
    elements, plus roundings 2^-22 / 2^-6 of the sums."""
    rows, d, step = 4, 96, 2.0 ** -6
    x, f, gate, w_post, w_pre = norm_inputs(rows, d, FP, "row", 3)
    g = gen(4)
    Gz, Gh = draw((rows, d), FP, g), draw((rows, d), FP, g)
    kw = dict(gate_kind="row", alpha=0.5)

    def loss(x, f, gate, w_post, w_pre):
        z, h, *_ = blk.norm_forward(x, f, gate, w_post, w_pre, **kw)
        return ((Gz * z).double().sum() + (Gh * h).double().sum()).item()

    z, _, rq, rp = blk.norm_forward(x, f, gate, w_post, w_pre, **kw)
    grads = blk.norm_backward(Gz, Gh, z, f, gate, w_post, w_pre, rq, rp, **kw)
    args = [x, f, gate, w_post, w_pre]
    for i, t in enumerate(grads):
        v = draw(args[i].shape, FP, g)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * v, args[i] - step * v
        num, want = (loss(*up) - loss(*down)) / (2 * step), (t.double() * v.double()).sum().item()
        assert abs(num - want) <= rows * d * (step ** 2 + 2.0 ** -16), (i, num, want)


# ---------------------------------------------------------------- embedding
EMBED = [(1, 1, 1), (1, 50, 64), (7, 3, 33), (64, 10, 128), (300, 1000, 72), (513, 97, 40), (2048, 5000, 24), (2049, 5000, 24),
         (5000, 70000, 16), (4097, 2, 264), (3000, 1, 8), (6000, 1100000, 3), (9000, 20000, 64),
         (9001, 300, 37), (65536, 131, 8), (65537, 3000, 8), (70001, 1100000, 5)]


@pytest.mark.parametrize("rows,V,d", EMBED)
@pytest.mark.parametrize("dtype,ids_dtype", [(BF, torch.int64), (HF, torch.int32), (FP, torch.int64)])
def test_embedding(blk, rows, V, d, dtype, ids_dtype):
    g = gen(rows + V)
    table, dout = draw((V, d), dtype, g), draw((rows, d), dtype, g)
    ids = (V * torch.rand(rows, generator=g, device="cuda") ** 3).long().clamp(max=V - 1)    # frequent low ids
    ids[torch.rand(rows, generator=g, device="cuda") < 0.1] = -1
    if rows > 4:
        ids[3] = V                                                                            # just past the table
        ids[4] = torch.iinfo(ids_dtype).min
    ids = ids.to(ids_dtype)
    out = blk.embed_forward(ids, table, scale=1.7)
    scale = float(np.float32(1.7))
    ref = ob.embed_forward(ids.cpu().numpy(), f64(table), scale)
    close(out, ref, np.abs(ref), 1)
    dt = blk.embed_backward(ids, dout, V, scale=1.7, dtable=torch.full((V, d), 5.0, dtype=dtype, device="cuda"))
    gref, size = ob.embed_backward(ids.cpu().numpy(), f64(dout), V, scale)
    most = int(torch.bincount(ids[(ids >= 0) & (ids < V)].long(), minlength=1).max()) if rows else 0
    close(dt, gref, size, most)
    assert torch.equal(dt, blk.embed_backward(ids, dout, V, scale=1.7))
    base = draw((V, d), FP, g)
    acc = base.clone()
    assert blk.embed_backward(ids, dout, V, scale=1.7, dtable=acc, accumulate=True) is acc
    close(acc, f64(base) + gref, size + np.abs(f64(base)), most + 1)
    untouched = torch.ones(V, dtype=torch.bool, device="cuda")
    untouched[ids[(ids >= 0) & (ids < V)].long()] = False
    assert torch.equal(acc[untouched], base[untouched])


def test_embedding_of_nothing_and_of_padding_only(blk):
    for ids in (torch.empty(0, dtype=torch.int64, device="cuda"), torch.full((5, 3), -1, dtype=torch.int32, device="cuda")):
        table = draw((9, 16), BF, gen(0))
        out = blk.embed_forward(ids, table)
        assert out.shape == (*ids.shape, 16) and torch.all(out == 0)
        g = blk.embed_backward(ids, out, 9, dtable=torch.ones((9, 16), dtype=BF, device="cuda"))
        assert torch.all(g == 0)


def test_embedding_strides(blk):
    g = gen(3)
    table, dout = draw((50, 48), BF, g)[:, 8:40], draw((70, 40), BF, g)[:, :32]
    ids = torch.randint(0, 50, (70,), generator=g, device="cuda")
    assert torch.equal(blk.embed_forward(ids, table), table[ids])
    grad = torch.zeros((50, 35), dtype=FP, device="cuda")
    blk.embed_backward(ids, dout, 50, dtable=grad[:, :32])
    ref, size = ob.embed_backward(ids.cpu().numpy(), f64(dout), 50)
    close(grad[:, :32], ref, size, 70)
    assert torch.all(grad[:, 32:] == 0)


def test_embedding_gradient_is_the_lookups_transpose(blk):
    """<G, out(table + v) - out(table - v)> / 2 = <dtable, v>: exact in small
    dyadic values."""
    g = gen(5)
    q = lambda *s: torch.randint(-8, 9, s, generator=g, device="cuda").float() / 8  # noqa: E731
    table, v, G = q(20, 24), q(20, 24), q(90, 24)
    ids = torch.randint(-1, 21, (90,), generator=g, device="cuda")
    f = lambda t: (G * blk.embed_forward(ids, t, scale=2.0)).double().sum().item()  # noqa: E731
    assert (f(table + v) - f(table - v)) / 2 == (blk.embed_backward(ids, G, 20, scale=2.0) * v).double().sum().item()


# ---------------------------------------------------------------- streams
def test_calls_run_on_the_given_stream(blk):
    g = gen(0)
    s = torch.cuda.Stream()
    x, w = draw((64, 64), BF, g), draw((2, 32, 64), BF, g)
    off = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    want = blk.grouped_forward(x, w, off)
    nz = blk.norm_forward(x, x, None, None, None)
    ids = torch.arange(64, device="cuda") % 20
    e, ge = blk.embed_forward(ids, x), blk.embed_backward(ids, x, 20)
    s.wait_stream(torch.cuda.current_stream())
    got = blk.grouped_forward(x, w, off, stream=s), blk.norm_forward(x, x, None, None, None, stream=s)
    ee, gg = blk.embed_forward(ids, x, stream=s), blk.embed_backward(ids, x, 20, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got[0], want) and all(torch.equal(a, b) for a, b in zip(got[1], nz))
    assert torch.equal(ee, e) and torch.equal(gg, ge)


def test_calls_are_captured_in_a_graph(blk):
    """One capture of every operator, replayed on new contents of its inputs."""
    g = gen(1)
    off = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
    x, dy, w = draw((300, 128), BF, g), draw((300, 64), BF, g), draw((3, 64, 128), BF, g)
    wn, ids = draw((128,), BF, g), torch.randint(0, 40, (300,), generator=g, device="cuda")

    def calls():
        z, h, rq, rp = blk.norm_forward(x, x, None, wn, wn)
        return (blk.grouped_forward(x, w, off), *blk.grouped_backward(dy, x, w, off), z, h,
                *(t for t in blk.norm_backward(h, z, z, x, None, wn, wn, rq, rp) if t is not None),
                blk.embed_forward(ids, x), blk.embed_backward(ids, x, 40))

    calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls()
    for seed in (5, 6):
        g = gen(seed)
        for t in (x, dy, w, wn):
            t.copy_(draw(t.shape, t.dtype, g))
        ids.copy_(torch.randint(-1, 41, (300,), generator=g, device="cuda"))
        off.copy_(torch.tensor([[0, 7, 250, 290], [3, 3, 200, 300]][seed - 5], dtype=torch.int32))
        graph.replay()
        for a, b in zip(out, calls()):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- offsets past 32 bits
def test_norm_past_32_bits(blk):
    rows, d = 270000, 8192          # 2.2e9 elements a tensor
    g = gen(2)
    x = torch.empty((rows, d), dtype=BF, device="cuda").normal_(generator=g)
    w = draw((d,), BF, g)
    z, h, rq, rp = blk.norm_forward(x, x, None, w, w, eps=1e-5)
    pick = torch.tensor([0, 1, 131071, 131072, 262143, 262144, 269999], device="cuda")
    o = ob.norm_forward(f64(x[pick]), f64(x[pick]), None, f64(w), f64(w), eps=1e-5)
    close(z[pick], o["z"], o["z_size"], d)
    close(h[pick], o["h"], o["h_size"] * 4, d)
    dx, df, _, _, _ = blk.norm_backward(x, h, z, x, None, w, w, rq, rp)
    ref, size = ob.norm_backward(*(f64(t[pick]) for t in (x, h, z, x)), None, f64(w), f64(w), f64(rq[pick]), f64(rp[pick]))
    close(dx[pick], ref["dx"], size["dx"], d)
    close(df[pick], ref["df"], size["df"], d)


def test_embedding_past_32_bits(blk):
    V, d, rows = 300000, 8192, 3000
    g = gen(3)
    table = torch.empty((V, d), dtype=BF, device="cuda").normal_(generator=g)
    ids = torch.randint(V - 1000, V, (rows,), generator=g, device="cuda")
    out = blk.embed_forward(ids, table)
    assert torch.equal(out, table[ids])
    grad = blk.embed_backward(ids, out, V, dtable=table.fill_(3.0))
    want = torch.zeros((1000, d), dtype=torch.float64, device="cuda").index_add_(0, ids - (V - 1000), out.double())
    size = torch.zeros((1000, d), dtype=torch.float64, device="cuda").index_add_(0, ids - (V - 1000), out.double().abs())
    close(grad[V - 1000:], f64(want), f64(size), 40)
    assert not grad[:V - 1000].any()


def test_grouped_past_32_bits(blk):
    rows, K, N = 270000, 8192, 64
    g = gen(4)
    x = torch.empty((rows, K), dtype=BF, device="cuda").normal_(generator=g)
    w = draw((2, N, K), BF, g, K ** -0.5)
    off = torch.tensor([0, 135000, rows], dtype=torch.int32, device="cuda")
    y = blk.grouped_forward(x, w, off)
    pick = torch.tensor([0, 134999, 135000, 262143, 262144, 269999], device="cuda")
    e = (pick >= 135000).long()
    ref = np.einsum("rk,rnk->rn", f64(x[pick]), f64(w[e]))
    size = np.einsum("rk,rnk->rn", np.abs(f64(x[pick])), np.abs(f64(w[e])))
    close(y[pick], ref, size, K)
    dx, _ = blk.grouped_backward(y, x, w, off, need_dw=False)
    close(dx[pick], np.einsum("rn,rnk->rk", f64(y[pick]), f64(w[e])), np.einsum("rn,rnk->rk", np.abs(f64(y[pick])), np.abs(f64(w[e]))), N)
    del dx, x, y
    # many experts: w itself past 32 bits, on few rows and on the tensor cores
    E, N, K = 600, 1024, 4096
    w = torch.empty((E, N, K), dtype=BF, device="cuda").normal_(generator=g)
    for rows in (8, 300):
        x = draw((rows, K), BF, g, K ** -0.5)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[E] = rows
        off[E - 1] = rows // 2
        y = blk.grouped_forward(x, w, off)
        for lo, hi, e in ((0, rows // 2, E - 2), (rows // 2, rows, E - 1)):
            close(y[lo:hi], f64(x[lo:hi]) @ f64(w[e]).T, np.abs(f64(x[lo:hi])) @ np.abs(f64(w[e])).T, K)


# ---------------------------------------------------------------- rows that share chunks, launches that overlap
@pytest.mark.parametrize("rows,d", [(2000, 515), (1700, 1027), (1100, 2883), (700, 4095), (700, 4604)])
@pytest.mark.parametrize("kind,post,pre", [("full", True, True), ("row", False, True), ("channel", True, False),
                                           ("none", False, False)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_many_rows_of_odd_width(blk, rows, d, kind, post, pre, dtype):
    check_norm(blk, rows, d, dtype, kind, post, pre, 0.75, seed=d)


@pytest.mark.parametrize("d", [515, 2883, 4095, 7167])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_neighbours_stay_apart(blk, d, dtype):
    """A row's chunks hold columns of the rows beside it: what is not finite there stays there."""
    rows = 700
    x, f, gate, w_post, w_pre = norm_inputs(rows, d, dtype, "full", 3)
    g = gen(4)
    dz, dh = draw((rows, d), dtype, g), draw((rows, d), dtype, g)
    kw = dict(gate_kind="full", alpha=0.5)

    def run(bad):
        t = [v.clone() for v in (x, f, gate, dz, dh)]
        if bad:
            for i, v in enumerate(t):
                v[1::2] = (float("nan"), float("inf"), float("-inf"))[i % 3]
        z, h, r_post, r_pre = blk.norm_forward(t[0], t[1], t[2], w_post, w_pre, **kw)
        dx, df, dg = blk.norm_backward(t[3], t[4], z, t[1], t[2], w_post, w_pre, r_post, r_pre, **kw)[:3]
        return [v[::2] for v in (z, h, r_post, r_pre, dx, df, dg)]

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


def test_overlapping_launches(blk):
    """Calls back to back, each read by a kernel right behind it, give what calls one at a time give."""
    g = gen(9)
    sizes = [(2043, 8, 512, 768), (900, 24, 128, 256), (3000, 5, 264, 520), (600, 300, 64, 72)]
    calls = []
    for rows, E, N, K in sizes:
        counts = split(rows, E, "skew", rows)
        counts[0], counts[-1] = 0, counts[-1] + counts[0]
        off = offsets_of(counts, 0)
        x, dy, w = draw((rows, K), BF, g), draw((rows, N), BF, g), draw((E, N, K), BF, g, K ** -0.5)
        calls.append(lambda dy=dy, x=x, w=w, off=off: blk.grouped_backward(dy, x, w, off))
    big = draw((64, 512, 768), BF, g)  # experts enough that those without rows are written apart
    few = torch.zeros(65, dtype=torch.int32)
    few[30:] = 700
    few = few.cuda()
    dy, x = draw((700, 512), BF, g), draw((700, 768), BF, g)
    calls.append(lambda: blk.grouped_backward(dy, x, big, few))
    for rows, V, d in [(515, 5001, 33), (5000, 700, 128), (70000, 300, 40)]:
        ids, dout = torch.randint(0, V, (rows,), generator=g, device="cuda"), draw((rows, d), BF, g)
        calls.append(lambda ids=ids, dout=dout, V=V: (blk.embed_backward(ids, dout, V),))
    for rows, d in [(700, 2883), (300, 9000), (40, 512)]:
        x_, f, gate, w_post, w_pre = norm_inputs(rows, d, BF, "channel", d)
        z, _, r_post, r_pre = blk.norm_forward(x_, f, gate, w_post, w_pre, gate_kind="channel")
        calls.append(lambda z=z, f=f, gate=gate, a=w_post, b=w_pre, p=r_post, q=r_pre, x_=x_: blk.norm_backward(
            x_, f, z, f, gate, a, b, p, q, gate_kind="channel"))
    alone = []
    for call in calls:
        out = call()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in out])
        torch.cuda.synchronize()
    for _ in range(4):
        copies = [[t.clone() for t in call()] for call in calls]
        for a, b in zip(alone, copies):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
