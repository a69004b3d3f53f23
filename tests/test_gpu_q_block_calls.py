"""GPU tests of calls around the layer in the places where their inputs, streams
and memory are not the usual ones."""
import numpy as np
import pytest
import torch

from oracle import block as ob

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


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


def spread(t):
    return torch.stack([t, t], -1).flatten()[::2]


def test_a_call_on_another_stream_does_not_wait_for_the_current_one(blk):
    """Inputs that the calls have to copy, on a side stream while the current one is
    busy: right results before the current stream is done."""
    g = gen(0)
    R, E, N, K, V = 200, 3, 72, 136, 50
    x, w, dy = turned(draw((R, K), BF, g)), turned(draw((E, N, K), BF, g)), draw((1, N), BF, g).expand(R, N)
    off = spread(torch.tensor([0, 30, 30, R], dtype=torch.int32, device="cuda"))
    f, gate, wq = turned(draw((R, K), BF, g)), turned(draw((R, K), BF, g)), spread(draw((K,), BF, g))
    ids, table = spread(torch.randint(-1, V, (R,), generator=g, device="cuda")), turned(draw((V, K), BF, g))
    z, _, rq, rp = blk.norm_forward(x, f, gate, wq, wq, gate_kind="full")
    z, rq, rp = turned(z), spread(rq), spread(rp)

    def calls(stream):
        return (blk.grouped_forward(x, w, off, stream=stream), *blk.grouped_backward(dy, x, w, off, stream=stream),
                *blk.norm_forward(x, f, gate, wq, wq, gate_kind="full", stream=stream),
                *blk.norm_backward(x, f, z, f, gate, wq, wq, rq, rp, gate_kind="full", stream=stream),
                blk.embed_forward(ids, table, stream=stream), blk.embed_backward(ids, x, V, stream=stream))

    want = calls(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    calls(side)                                 # its memory and kernels are there from here on
    torch.cuda.synchronize()
    busy, done = torch.cuda.Event(), torch.cuda.Event()
    torch.cuda._sleep(1_000_000_000)            # about half a second
    busy.record()
    got = calls(side)
    done.record(side)
    done.synchronize()
    assert not busy.query()
    with torch.cuda.stream(side):
        same = [torch.equal(a, b) for a, b in zip(got, want)]
    assert len(got) == len(want) and all(same)
    by_handle = calls(side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(by_handle, want))


# ---------------------------------------------------------------- what is not finite, and the ends of the range
def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


U = {BF: 2.0 ** -8, HF: 2.0 ** -11, FP: 2.0 ** -24}


def near(got, ref, size, n):
    """Equal where the reference is not finite; elsewhere within a rounding of the output's
    type and (n + 32) 2^-22 of the terms' sizes, as in test_gpu_o_block.py."""
    got_, fin = f64(got), np.isfinite(ref)
    assert np.array_equal(got_[~fin], ref[~fin], equal_nan=True)
    tol = U[got.dtype] * np.abs(ref[fin]) + (n + 32) * 2.0 ** -22 * size[fin] + 2.0 ** -25
    assert np.all(np.abs(got_[fin] - ref[fin]) <= tol)


# both register kernels, rows in flight through shared memory (even and odd), long rows
NORM_PATHS = [(37, 200), (37, 264), (37, 1027), (333, 1032), (311, 1027), (5, 9000), (5, 9001)]


@pytest.mark.parametrize("kind", ["none", "channel", "row", "full"])
@pytest.mark.parametrize("rows,d", NORM_PATHS)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_gradient_of_an_infinite_block_output_without_its_norm(blk, rows, d, kind, dtype):
    """df = g t takes nothing from f, and without the pre norm t = dz: what f holds does not matter to df,
    and a gate's gradient sum t f is infinite only where its own terms are."""
    g = gen(d)
    x, f, dz, dh = (draw((rows, d), dtype, g) for _ in range(4))
    f[1, 3], f[2, d - 1], f[4, d // 2] = float("inf"), float("-inf"), float("nan")
    shape = {"none": None, "channel": (d,), "row": (rows,), "full": (rows, d)}[kind]
    gate = None if shape is None else draw(shape, dtype, g)
    kw = dict(gate_kind=kind, post=False, pre=False, alpha=0.5)
    got = blk.norm_backward(dz, None, None, f, gate, **kw)
    with np.errstate(invalid="ignore"):
        ref, size = ob.norm_backward(f64(dz), None, None, f64(f), f64(gate), None, None, None, None, kind, False, False, 0.5)
    assert np.all(np.isfinite(ref["df"]))
    for name, t in zip(("dx", "df", "dgate"), got):
        assert (t is None) == (ref[name] is None)
        if t is not None:
            near(t, ref[name], size[name], d + rows)
    # with the pre norm (over a z that is finite)
    w_pre, r = draw((d,), dtype, g), (1 + draw((rows,), FP, g).abs())
    dx, df, _, _, dw = blk.norm_backward(dz, dh, x, f, gate, None, w_pre, None, r, gate_kind=kind, post=False, alpha=0.5)
    with np.errstate(invalid="ignore"):
        ref, size = ob.norm_backward(f64(dz), f64(dh), f64(x), f64(f), f64(gate), None, f64(w_pre), None, f64(r), kind, False,
                                     True, 0.5)
    for name, t in (("dx", dx), ("df", df), ("dw_pre", dw)):
        assert np.all(np.isfinite(ref[name]))
        near(t, ref[name], size[name], d + rows)


@pytest.mark.parametrize("rows,d", NORM_PATHS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("size", [2.0 ** 47, 2.0 ** -47])
def test_norm_gradients_of_large_and_small_rows(blk, rows, d, dtype, size):
    """rms(f) and rms(z) whose cubes leave fp32 while their squares do not: all gradients, relative to their
    own terms (df and dx are of the size of t / rms)."""
    g = gen(d + 1)
    f, z, dz, dh = draw((rows, d), dtype, g, size), draw((rows, d), dtype, g, size), draw((rows, d), dtype, g, 1 / size), \
        draw((rows, d), dtype, g)
    wq, wp, gate = draw((d,), dtype, g), draw((d,), dtype, g), draw((rows,), dtype, g)
    rq, rp = (torch.rsqrt(t.double().square().mean(1)).float() for t in (f, z))
    got = blk.norm_backward(dz, dh, z, f, gate, wq, wp, rq, rp, gate_kind="row")
    ref, sz = ob.norm_backward(*(f64(t) for t in (dz, dh, z, f, gate, wq, wp, rq, rp)), kind="row")
    for name, t in zip(("dx", "df", "dgate", "dw_post", "dw_pre"), got):
        tol = U[dtype] * np.abs(ref[name]) + (d + rows + 32) * 2.0 ** -22 * sz[name]
        assert np.all(np.isfinite(f64(t))) and np.all(np.abs(f64(t) - ref[name]) <= tol), name


# ---------------------------------------------------------------- memory
def test_gradients_of_narrow_slices(blk):
    """A few columns of a wide buffer: the gradients of the same columns by themselves."""
    g = gen(3)
    R, E, N, K = 300, 3, 64, 72
    x, f, gate = (draw((R, 16 * K), BF, g)[:, i * K:(i + 1) * K] for i in (0, 1, 15))
    dy, w, v = draw((R, N), BF, g), draw((E, N, K), BF, g), draw((K,), BF, g)
    off = torch.tensor([0, 100, 100, R], dtype=torch.int32, device="cuda")
    z, dz, dh = (draw((R, K), BF, g) for _ in range(3))
    r = torch.rand(R, generator=g, device="cuda") + 0.5
    got = (*blk.grouped_backward(dy, x, w, off), *blk.norm_backward(dz, dh, z, f, gate, v, v, r, r, gate_kind="full"))
    c = [t.contiguous() for t in (x, f, gate)]
    want = (*blk.grouped_backward(dy, c[0], w, off), *blk.norm_backward(dz, dh, z, c[1], c[2], v, v, r, r, gate_kind="full"))
    assert len(got) == 7 and all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(t.untyped_storage().nbytes() <= t.numel() * t.element_size() for t in got)


def test_embedding_of_a_single_id_trains(blk):
    from mixture_experts_layer_device_gb300.module import TokenEmbedding
    m = TokenEmbedding(7, 24, scale=2.0)
    y = m(torch.tensor(3, device="cuda"))
    assert torch.equal(y, 2.0 * m.weight[3])
    y.sum().backward()
    want = torch.zeros_like(m.weight)
    want[3] = 2.0
    assert torch.equal(m.weight.grad, want)


# ---------------------------------------------------------------- outputs in their inputs' place
@pytest.mark.parametrize("kind", ["none", "channel", "row", "full"])
@pytest.mark.parametrize("rows,d", [(40, 200), (40, 4096), (40, 2883), (700, 2883), (700, 4096), (2000, 515), (170, 13000)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_backward_in_place(blk, rows, d, kind, dtype):
    """dx in dz's buffer and df in f's, as the boundary allows: the numbers of separate buffers."""
    import mixture_experts_layer_device_gb300 as pkg
    g = gen(rows + d)
    dz, dh, z, f = (draw((rows, d), dtype, g) for _ in range(4))
    shape = {"none": None, "channel": (d,), "row": (rows,), "full": (rows, d)}[kind]
    gate = None if shape is None else draw(shape, dtype, g)
    wq, wp = draw((d,), dtype, g), draw((d,), dtype, g)
    rq, rp = (torch.rand(rows, generator=g, device="cuda") + 0.5 for _ in range(2))
    want = blk.norm_backward(dz, dh, z, f, gate, wq, wp, rq, rp, gate_kind=kind, alpha=0.5)
    cfg = pkg.MoeNormConfig(rows, d, {BF: 0, FP: 2}[dtype], 3, pkg.GATES[kind], 0.5, 0.0, 0, 0, 0, 0, 0)
    ws = torch.empty(pkg.moe_norm_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    dg, dwq, dwp = None if gate is None else torch.empty_like(gate), torch.empty_like(wq), torch.empty_like(wp)
    pkg.check(pkg.moe_norm_backward(cfg, dz, dh, z, f, gate, wq, wp, rq, rp, dz, f, dg, dwq, dwp, ws))
    for a, b in zip((dz, f, dg, dwq, dwp), want):
        assert a is b or torch.equal(a, b)


@pytest.mark.parametrize("rows,d", [(40, 200), (40, 4096), (700, 2883), (700, 4096), (170, 20000)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_forward_into_the_residual_stream(blk, rows, d, dtype):
    """z in x's buffer: the residual stream updated where it lies."""
    g = gen(rows + d)
    x, f, w = draw((rows, d), dtype, g), draw((rows, d), dtype, g), draw((d,), dtype, g)
    want = blk.norm_forward(x, f, None, w, w)
    got = blk.norm_forward(x, f, None, w, w, z=x)
    assert got[0] is x and all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------- rows where the kernels change
def products(blk, x, w, off):
    with np.errstate(invalid="ignore"):
        ref, size = ob.grouped_forward(f64(x), f64(w), off.cpu().numpy())
    near(blk.grouped_forward(x, w, off), ref, size, x.shape[1])


@pytest.mark.parametrize("rows", [1, 5, 64, 65])
@pytest.mark.parametrize("at", [0, 17, 39])
def test_grouped_all_rows_on_one_of_many_experts(blk, rows, at):
    """The streaming kernel's rule looks at the average; all rows may be one expert's."""
    g = gen(rows)
    x, w = draw((rows, 136), BF, g), draw((40, 200, 136), BF, g)
    off = torch.zeros(41, dtype=torch.int32, device="cuda")
    off[at + 1:] = rows
    products(blk, x, w, off)


@pytest.mark.parametrize("shift", [1, 4, 8])
@pytest.mark.parametrize("which", ["x", "w", "dy", "all"])
def test_grouped_operands_off_16_bytes(blk, which, shift):
    """Row strides that are whole 16-byte pieces, and rows that start inside one."""
    g = gen(shift)
    R, E, N, K = 400, 4, 128, 256
    off = torch.tensor([0, 100, 100, 333, 398], dtype=torch.int32, device="cuda")

    def make(name, *shape):
        cut = which in (name, "all")
        t = draw((*shape[:-1], shape[-1] + 16), BF, g)
        return t[..., shift:shift + shape[-1]] if cut else t[..., :shape[-1]].contiguous()

    x, w, dy = make("x", R, K), make("w", E, N, K), make("dy", R, N)
    products(blk, x, w, off)
    dx, dw = blk.grouped_backward(dy, x, w, off)
    rx, rw, sx, sw = ob.grouped_backward(f64(dy), f64(x), f64(w), off.cpu().numpy())
    near(dx, rx, sx, N)
    near(dw, rw, sw, 233)
