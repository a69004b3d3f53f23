"""The operators that end a training step where their values leave the ordinary
range, against the definitions (exact values where the inputs make them so)."""
import math

import pytest
import torch

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
