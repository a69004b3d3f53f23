"""CPU-only checks of what block.py does around the library's calls: in which
stream's order its copies, allocations and launches stand, which GPUs its
tensors are on, what it allocates.  CPU tensors pose as GPU tensors, and a
stand-in for the library records its calls."""
import contextlib
import types

import pytest
import torch

from mixture_experts_layer_device_gb300 import block

BF = torch.bfloat16


class Gpu(torch.Tensor):
    """A CPU tensor that says it is on GPU 0 and records what is done with it."""
    log, index = [], 0
    is_cuda = property(lambda t: True)
    device = property(lambda t: torch.device("cuda", t.index))

    def get_device(t):
        return t.index

    def data_ptr(t):
        return 1 << 12

    def contiguous(t):
        if t.is_contiguous():
            return t
        Gpu.log.append(("copy", torch.cuda.current_stream()))
        return super().contiguous()

    def reshape(t, *shape):
        r = super().reshape(*shape)
        if r.untyped_storage().data_ptr() != t.untyped_storage().data_ptr():
            Gpu.log.append(("copy", torch.cuda.current_stream()))
        return r

    def record_stream(t, stream):
        Gpu.log.append(("kept", stream, t.untyped_storage().data_ptr()))


class OtherGpu(Gpu):
    index = 1


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


MAIN, SIDE = Stream(11), Stream(22)


class Library:
    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_bytes"):
                return 512
            Gpu.log.append(("launch", name, args[-1]))
            return 0
        return call


@pytest.fixture
def gpu(monkeypatch):
    """The recorded calls; `gpu.current` is the current GPU's index."""
    state = types.SimpleNamespace(log=[], stream=MAIN, current=0, allocated=0)
    Gpu.log = state.log

    @contextlib.contextmanager
    def within(stream):
        before, state.stream = state.stream, stream
        yield
        state.stream = before

    def stand_in(make):
        def call(*args, device=None, **kw):
            state.log.append(("new", state.stream))
            t = make(*args, **kw).as_subclass(Gpu)
            state.allocated = max(state.allocated, t.untyped_storage().nbytes())
            return t
        return call

    monkeypatch.setattr(torch, "empty", stand_in(torch.empty))
    monkeypatch.setattr(torch.cuda, "stream", within)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state.stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: {11: MAIN, 22: SIDE}[handle])
    monkeypatch.setattr(block, "_stream", lambda s: s if isinstance(s, int) else (s or state.stream).cuda_stream)
    monkeypatch.setattr(block, "lib", Library)
    monkeypatch.setattr(block, "_current_gpu", lambda: state.current, raising=False)
    plans = (block._grouped_plan, block._norm_plan, block._embed_plan)
    for p in plans:
        p.cache_clear()
    yield state
    for p in plans:
        p.cache_clear()


def on(kind, *shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype).as_subclass(kind)


def crooked(kind, *shape, dtype=BF):
    """The same whose last two dimensions lie in the other order: the call copies it."""
    return on(kind, *shape[:-2], shape[-1], shape[-2], dtype=dtype).transpose(-1, -2)


def spread(kind, n, dtype):
    return on(kind, 2 * n, dtype=dtype)[::2]


def calls(make, vec):
    """(operator, its tensors, its options): matrices by make(*shape), vectors by vec(n, dtype)."""
    R, E, N, K, V = 6, 3, 4, 5, 7
    x, w, off, dy = make(R, K), make(E, N, K), vec(E + 1, torch.int32), make(R, N)
    f, g, wq, r, ids = make(R, K), make(R, K), vec(K, BF), vec(R, torch.float32), vec(R, torch.int64)
    return [
        (block.grouped_forward, dict(x=x, w=w, offsets=off), {}),
        (block.grouped_backward, dict(dy=dy, x=x, w=w, offsets=off), {}),
        (block.norm_forward, dict(x=x, f=f, gate=g, w_post=wq, w_pre=wq), dict(gate_kind="full")),
        (block.norm_backward, dict(dz=x, dh=f, z=f, f=f, gate=g, w_post=wq, w_pre=wq, r_post=r, r_pre=r),
         dict(gate_kind="full")),
        (block.embed_forward, dict(ids=ids, table=make(V, K)), {}),
        (block.embed_backward, dict(ids=ids, dout=x), dict(V=V)),
    ]


CALLS = ["grouped_forward", "grouped_backward", "norm_forward", "norm_backward", "embed_forward", "embed_backward"]


@pytest.mark.parametrize("i", range(6), ids=CALLS)
@pytest.mark.parametrize("given", [None, SIDE, 22], ids=["current", "stream", "handle"])
def test_copies_and_memory_belong_to_the_stream_of_the_launch(gpu, i, given):
    fn, tensors, opts = calls(lambda *s: crooked(Gpu, *s), lambda n, dt: spread(Gpu, n, dt))[i]
    out = fn(**tensors, **opts, stream=given)
    stream = MAIN if given is None else SIDE
    launches = [e for e in gpu.log if e[0] == "launch"]
    assert len(launches) == 1 and launches[0][2] == stream.cuda_stream
    made = [e for e in gpu.log if e[0] in ("copy", "new")]
    assert {e[0] for e in made} == {"copy", "new"}
    assert all(e[1] is stream for e in made), made
    assert gpu.stream is MAIN
    if given is not None:       # the caller's tensors outlive their use there, the results theirs on the caller's stream
        kept = {e[1:] for e in gpu.log if e[0] == "kept"}
        for t in tensors.values():
            assert (SIDE, t.untyped_storage().data_ptr()) in kept
        for t in out if isinstance(out, tuple) else (out,):
            if t is not None:
                assert (MAIN, t.untyped_storage().data_ptr()) in kept


@pytest.mark.parametrize("i", range(6), ids=CALLS)
def test_tensors_on_another_gpu_are_refused(gpu, i):
    """All on the current GPU, or a ValueError before anything is launched."""
    fn, tensors, opts = calls(lambda *s: on(Gpu, *s), lambda n, dt: on(Gpu, n, dtype=dt))[i]
    fn(**tensors, **opts)
    assert len([e for e in gpu.log if e[0] == "launch"]) == 1
    for name, t in tensors.items():
        with pytest.raises(ValueError):
            fn(**{**tensors, name: t.as_subclass(OtherGpu)}, **opts)
        with pytest.raises(ValueError):
            fn(**{**tensors, name: t.as_subclass(torch.Tensor)}, **opts)
    with pytest.raises(ValueError):
        fn(**{k: t.as_subclass(OtherGpu) for k, t in tensors.items()}, **opts)
    outputs = {"grouped_forward": dict(out=(6, 4)), "grouped_backward": dict(dx=(6, 5), dw=(3, 4, 5)),
               "norm_forward": dict(z=(6, 5), h=(6, 5)), "embed_forward": dict(out=(6, 5)),
               "embed_backward": dict(dtable=(7, 5))}
    for name, shape in outputs.get(CALLS[i], {}).items():
        fn(**tensors, **opts, **{name: on(Gpu, *shape)})
        with pytest.raises(ValueError):
            fn(**tensors, **opts, **{name: on(OtherGpu, *shape)})
    assert len([e for e in gpu.log if e[0] == "launch"]) == 1 + len(outputs.get(CALLS[i], {}))
    gpu.current = 1
    with pytest.raises(ValueError):
        fn(**tensors, **opts)


def test_gradients_of_narrow_slices_take_no_wide_memory(gpu):
    """A gradient of a few columns of a wide buffer is not as wide as the buffer; one of a part
    of a fused buffer shares its stride, without a copy."""
    R, E, N, K = 64, 2, 40, 48

    def backward(wide):
        x, f, gate = (on(Gpu, R, wide * K)[:, :K] for _ in range(3))
        dy, z, v, r = on(Gpu, R, N), on(Gpu, R, K), on(Gpu, K), on(Gpu, R, dtype=torch.float32)
        gpu.log.clear()
        gpu.allocated = 0
        dx, dw = block.grouped_backward(dy, x, on(Gpu, E, N, K), on(Gpu, E + 1, dtype=torch.int32), need_dw=False)
        assert dx.shape == (R, K) and dw is None
        out = block.norm_backward(z, z, z, f, gate, v, v, r, r, gate_kind="full")
        assert all(t.shape == (R, K) for t in out[:3])
        return sum(e[0] == "copy" for e in gpu.log)

    assert backward(64) == 3 and gpu.allocated <= 2 * R * K * 2
    assert backward(8) == 0 and gpu.allocated <= 8 * R * K * 2


def test_an_embedding_of_one_id(gpu):
    """ids of any shape, a single one without a dimension among them, in both directions."""
    ids, table = torch.tensor(3).as_subclass(Gpu), on(Gpu, 7, 5)
    out = block.embed_forward(ids, table)
    assert out.shape == (5,)
    assert block.embed_backward(ids, out, 7).shape == (7, 5)
    with pytest.raises(ValueError):
        block.embed_backward(on(Gpu, 2, dtype=torch.int64), out, 7)


def test_status_texts_hold_for_every_entry_point():
    """The grouped products report offsets out of range in every build, and around the
    layer a pointer needs its element's alignment only."""
    from mixture_experts_layer_device_gb300 import STATUS, build, lib
    build.build()
    for code in (-3, -7):
        text = lib().moe_status_string(code).decode()
        assert text == STATUS[code] and "debug" not in text and "16" not in text


def test_numbers_are_read_at_every_call(gpu, monkeypatch):
    """alpha, eps and scale given as tensors that change in place: nothing is kept by which object came."""
    seen = []

    class Reading(Library):
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("workspace_bytes"):
                    return 512
                cfg = args[0]._obj
                seen.append((cfg.alpha, cfg.eps) if "norm" in name else cfg.scale)
                return 0
            return call

    monkeypatch.setattr(block, "lib", Reading)
    x, ids, number = on(Gpu, 6, 5), on(Gpu, 6, dtype=torch.int64), torch.tensor(0.5)
    r = on(Gpu, 6, dtype=torch.float32)
    for value in (0.5, 0.25):
        number.fill_(value)
        seen.clear()
        block.norm_forward(x, x, alpha=number, eps=number)
        block.norm_backward(x, x, x, x, r_post=r, r_pre=r, alpha=number)
        block.embed_forward(ids, x, scale=number)
        block.embed_backward(ids, x, 7, scale=number)
        assert seen == [(value, value), (value, 0.0), value, value]
