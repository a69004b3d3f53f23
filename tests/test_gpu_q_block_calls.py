"""GPU tests of calls around the layer in the places where their inputs, streams
and memory are not the usual ones."""
import pytest
import torch

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
