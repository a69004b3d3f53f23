"""Trains a small mixture-of-experts token model with everything the library has
around the layer: embedding -> [norm -> MoE layer -> norm, gate, residual] ->
[ragged experts of another activation -> norm, gate, residual] -> logits.

Block 1 is the MoE layer itself (router, SwiGLU experts).  Block 2 is built by
hand from moe_route's offsets and two GroupedLinear maps with a squared ReLU
between them: experts of the user's own.  The task is to name the token itself,
so the loss falls from log V as the model learns to pass it on.

    python examples/block_training.py [--steps 60] [--tokens 512]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_layer_device_gb300 as moe_lib  # noqa: E402
from mixture_experts_layer_device_gb300.module import BlockNorm, GroupedLinear, MoE, TokenEmbedding  # noqa: E402


class RaggedExperts(torch.nn.Module):
    """Top-k experts with a squared ReLU: W_2 relu(W_1 x)^2, on the rows that
    moe_route sorts by expert, without padding."""

    def __init__(self, T, d, m, E, k):
        super().__init__()
        self.router = torch.nn.Linear(d, E, bias=False, dtype=torch.bfloat16, device="cuda")
        self.up, self.down = GroupedLinear(E, m, d), GroupedLinear(E, d, m)
        self.cfg = moe_lib.config(T, 256, 128, E, k)
        self.T, self.E, self.k = T, E, k

    def forward(self, x):
        T, E, k = self.T, self.E, self.k
        logits = self.router(x).float()
        i32 = dict(dtype=torch.int32, device=x.device)
        idx, counts, offsets, perm = (torch.empty(n, **i32) for n in ((T, k), (E,), (E + 1,), (T * k,)))
        w = torch.empty((T, k), dtype=torch.float32, device=x.device)
        moe_lib.check(moe_lib.moe_route_noalloc(self.cfg, logits.detach(), idx, w, counts, offsets, perm))
        slot_of_row = torch.empty_like(perm)
        slot_of_row[perm.long()] = torch.arange(T * k, **i32)
        rows = x[(slot_of_row // k).long()]
        h = torch.relu(self.up(rows, offsets)).square()
        o = self.down(h, offsets)[perm.long()].view(T, k, -1)
        # the router learns through its softmax over the chosen logits (the kernel's w)
        w = torch.softmax(logits.gather(1, idx.long()), 1)
        return (w.unsqueeze(-1).to(o.dtype) * o).sum(1)


class Model(torch.nn.Module):
    def __init__(self, T, V=997, d=256, m=128, E=8, k=2):
        super().__init__()
        self.embed = TokenEmbedding(V, d, scale=math.sqrt(d))
        self.first = BlockNorm(d, post=False, pre=True)                       # h = norm(x)
        self.moe = MoE(T, d, m, E, k, fmt="bf16", router=True)
        self.between = BlockNorm(d, post=True, pre=True, gate="channel")       # x + g norm(f), and the next norm
        self.experts = RaggedExperts(T, d, m, E, k)
        self.last = BlockNorm(d, post=True, pre=True, gate="channel")
        self.head = GroupedLinear(1, V, d)                                     # logits: one group of all tokens
        self.all_rows = torch.tensor([0, T], dtype=torch.int32, device="cuda")

    def forward(self, ids):
        x = self.embed(ids)
        _, h = self.first(x)
        x, h = self.between(x, self.moe(h))
        _, h = self.last(x, self.experts(h))
        return self.head(h, self.all_rows)


def train(steps=60, tokens=512, lr=0.002, seed=0, say=print):
    """Losses of `steps` steps of Adam on fp32 masters."""
    torch.manual_seed(seed)
    model = Model(tokens)
    V = model.embed.weight.shape[0]
    params = list(model.parameters())
    masters = [p.detach().float() for p in params]
    opt = torch.optim.Adam([m.requires_grad_() for m in masters], lr=lr)
    losses = []
    for step in range(steps):
        ids = torch.randint(0, V // 8, (tokens,), device="cuda")
        ids[:: 17] = -1                                                        # padding
        loss = torch.nn.functional.cross_entropy(model(ids).float(), ids, ignore_index=-1)
        loss.backward()
        with torch.no_grad():
            for p, m in zip(params, masters):
                m.grad = None if p.grad is None else p.grad.float()
                p.grad = None
            opt.step()
            for p, m in zip(params, masters):
                p.copy_(m)
        losses.append(float(loss.detach()))
        if step % 10 == 0 or step == steps - 1:
            say("step %3d  loss %.4f" % (step, losses[-1]))
    return losses


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--steps", type=int, default=60)
    a.add_argument("--tokens", type=int, default=512)
    a = a.parse_args()
    train(a.steps, a.tokens)
