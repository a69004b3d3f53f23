"""Cases, plain forms and exact values of a training step's operators next to
the MoE layer: the loss over a vocabulary taken straight from the last hidden
rows, the gated products of a feed-forward block grouped by expert, and the
global norm of all gradients with their clipping.

`run` computes a case in its plain form (elementary torch operations in fp32,
rounded once), or through this package's kernels where `own` is true; `exact`
gives the same outputs in 64 bits from the definitions.

  vocab      z_t = W x_t,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t[y_t];
             dz_tv = (dloss_t + dlse_t) exp(z_tv - lse_t) - dloss_t [v = y_t],
             dx_t = sum_v dz_tv W_v,  dW_v = sum_t dz_tv x_t;
             a row whose label lies outside the vocabulary: all zeros
  gated      g = W_g x, u = W_u x, h = act(g) u for the rows of every expert;
             dg = dh u act'(g), du = dh act(g), dx = W_g^T dg + W_u^T du,
             dW = [dg, du]^T x; rows of no expert give 0
  grad       norm = sqrt(sum of all squares), c = min(1, max_norm / (norm + eps)),
             every gradient times c, in place or into fp32 masters' gradients
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # scoring the last five positions of a request against a large vocabulary (Kimi-K2.7 width):
        # the weights are read once
        dict(name="vocab_fwd_few", op="vocab_fwd", rows=5, V=131072, d=7168, ignored=0.0, weights="mean", dtype="bf16"),
        # the loss of a training step's 16,384 tokens, a few of them padding
        dict(name="vocab_fwd_sequence", op="vocab_fwd", rows=16384, V=131072, d=4096, ignored=0.03, weights="mean",
             dtype="bf16"),
        # the gradients of a fine-tuning step: prompts (nearly a third) are not trained on
        dict(name="vocab_bwd_sequence", op="vocab_bwd", rows=8192, V=131072, d=4096, ignored=0.3, weights="mean",
             dtype="bf16"),
        # a small model at odd sizes, weighted tokens and a penalty on the log-sum
        dict(name="vocab_bwd_odd", op="vocab_bwd", rows=515, V=50001, d=321, ignored=0.1, weights="weighted",
             dtype="fp16"),
        # one generated token through the gate/up product of a layer with 512 experts, top 10 (the
        # layer's Qwen3.5-397B-A17B shape)
        dict(name="gated_fwd_one_token", op="gated_fwd", rows=10, E=512, active=10, m=1024, K=4096, spread=0.0,
             outside=0, act="silu", save=False, dtype="bf16"),
        # the gate/up product of a training step of the same layer: 8192 tokens, top 10
        dict(name="gated_fwd_sequence", op="gated_fwd", rows=81920, E=512, active=512, m=1024, K=4096, spread=0.3,
             outside=0, act="silu", save=True, dtype="bf16"),
        # its gradients at another layer's width, with skewed loads and four idle experts
        dict(name="gated_bwd_skewed", op="gated_bwd", rows=32768, E=64, active=60, m=2048, K=7168, spread=1.2,
             outside=0, act="silu", dtype="bf16"),
        # a small dense block with another activation, some rows left out
        dict(name="gated_bwd_small", op="gated_bwd", rows=2043, E=1, active=1, m=1537, K=768, spread=0.0, outside=3,
             act="gelu", dtype="fp16"),
        # all gradients of a small model: many short tensors, latency counts
        dict(name="grad_norm_many", op="grad_norm", n=400, total=4000001, dtype="mixed"),
        # the expert weights of a large layer
        dict(name="grad_norm_experts", op="grad_norm", n=6, total=2818572288, dtype="bf16"),
        # a step's gradients clipped into the fp32 gradients that the optimizer's masters take
        dict(name="grad_clip_masters", op="grad_clip", n=120, total=300000007, place="masters", limit=0.25,
             dtype="bf16"),
        # in place, a quiet step: the norm stays below the limit
        dict(name="grad_clip_quiet", op="grad_clip", n=64, total=50331648, place="here", limit=2.0, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size over [lo, hi] by its logarithm: a multiple of 64, a multiple of 8, or any."""
    n, kind = _log(rng, lo, hi), rng.random()
    if kind < 0.5:
        n = max(64, n // 64 * 64)
    elif kind < 0.75:
        n = max(8, n // 8 * 8)
    return min(n, hi)


def draw(rng):
    op = rng.choice(["vocab_fwd", "vocab_bwd", "gated_fwd", "gated_bwd", "grad_norm", "grad_clip"])
    if op.startswith("vocab"):
        most = 16384 * 131072 * 4096 if op == "vocab_fwd" else 8192 * 131072 * 4096
        while True:
            c = dict(op=op, rows=_log(rng, 1, 16384), V=_log(rng, 100, 131072), d=_size(rng, 16, 8192),
                     ignored=rng.choice([0.0, 0.05, 0.5]), weights=rng.choice(["mean", "weighted"]),
                     dtype=rng.choice(["bf16", "bf16", "fp16"]))
            if c["rows"] * c["V"] * c["d"] <= most and c["V"] * c["d"] <= 131072 * 7168:
                return c
    if op.startswith("gated"):
        most = {"gated_fwd": 81920 * 1024 * 4096, "gated_bwd": 32768 * 2048 * 7168}[op]
        while True:
            E = _log(rng, 1, 512)
            c = dict(op=op, rows=_log(rng, 1, 81920), E=E, active=0, m=_size(rng, 8, 4096), K=_size(rng, 16, 7168),
                     spread=rng.choice([0.0, 0.4, 1.0]), outside=rng.choice([0, 0, 3]),
                     act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]),
                     dtype=rng.choice(["bf16", "bf16", "fp16"]))
            if op == "gated_fwd":
                c["save"] = rng.random() < 0.6
            c["active"] = min(c["rows"], max(1, round(E * rng.uniform(0.5, 1.0))))
            if c["rows"] * c["m"] * c["K"] <= most and c["active"] * c["m"] * c["K"] <= most // 160:
                return c
    while True:
        c = dict(op=op, n=_log(rng, 1, 500), total=_log(rng, 1000, 2800000000),
                 dtype=rng.choice(["bf16", "fp16", "fp32", "mixed"]))
        if op == "grad_clip":
            c["place"], c["limit"] = rng.choice([("masters", 0.1), ("masters", 3.0), ("apart", 0.5), ("here", 2.0)])
        size = _BYTES.get(c["dtype"], 2) + (0 if op == "grad_norm" or c["place"] == "here" else
                                            4 if c["place"] == "masters" else _BYTES.get(c["dtype"], 2))
        if c["total"] >= 8 * c["n"] and c["total"] * size <= 2818572288 * 2:
            return c


# ---------------------------------------------------------------- inputs
def _counts(case, g):
    """Rows of every expert: `active` experts, chosen by the seed, share the
    rows with log-normal weights of sigma `spread`, one row each at least."""
    E, active = case["E"], case["active"]
    rows = max(active, case["rows"] - case["outside"])
    weight = torch.exp(case["spread"] * torch.randn(active, generator=g, dtype=torch.float64))
    share = torch.floor(weight / weight.sum() * (rows - active)).to(torch.int64) + 1
    share[int(torch.argmax(weight))] += rows - int(share.sum())
    counts = torch.zeros(E, dtype=torch.int64)
    counts[torch.randperm(E, generator=g)[:active]] = share
    return counts.tolist()


def _normal(shape, std, dtype, gen):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, std, generator=gen)


def _flats(case):
    """(type, elements, tensors) of the buffers that hold the gradients: one of the
    case's type, or matrices in bf16 and a sixteenth of the elements in fp32."""
    n, total = case["n"], case["total"]
    if case["dtype"] != "mixed":
        return [(case["dtype"], total, n)]
    if n == 1:
        return [("bf16", total, 1)]
    return [("bf16", total - total // 16, n - n // 2), ("fp32", total // 16, n // 2)]


def _lengths(total, n, g):
    """n lengths of log-normal size that make up `total`, one at least each."""
    weight = torch.exp(1.5 * torch.randn(n, generator=g, dtype=torch.float64))
    part = torch.floor(weight / weight.sum() * (total - n)).to(torch.int64) + 1
    part[0] += total - int(part.sum())
    return part.tolist()


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=dict(case))
    if case["op"].startswith("vocab"):
        T, V, d, dt = case["rows"], case["V"], case["d"], _DT[case["dtype"]]
        s["w"] = _normal((V, d), d ** -0.5, dt, gen)
        # token frequencies fall as 1 / rank, ranks spread over the vocabulary
        u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64)
        rank = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
        labels = torch.randperm(V, generator=gen, device="cuda")[rank]
        # hidden rows that lean towards their token's weights, from not at all to surely
        x = torch.randn((T, d), generator=gen, device="cuda")
        lean = 12.0 * torch.rand((T, 1), generator=gen, device="cuda")
        x += lean * s["w"][labels].float()
        s["x"] = x.to(dt)
        out = torch.rand(T, generator=gen, device="cuda") < case["ignored"]
        labels[out] = -100
        s["x"][out] = math.nan        # what stands in rows that are left out does not count
        s["labels"] = labels
        if case["op"] == "vocab_bwd":
            keep = (labels >= 0).float()
            # the mean over the tokens that count; half precision is trained with a scaled loss
            s["dloss"] = keep * (4096.0 if case["dtype"] == "fp16" else 1.0) / keep.sum().clamp(min=1.0)
            if case["weights"] == "weighted":
                s["dloss"] *= 0.5 + torch.rand(T, generator=gen, device="cuda")
            # what the forward left
            s["lse"] = torch.zeros(T, device="cuda")
            w = s["w"].float()
            for rows in torch.nonzero(keep)[:, 0].split(4096):
                s["lse"][rows] = torch.logsumexp(s["x"][rows].float() @ w.T, 1)
            # a penalty 1e-4 lse^2 on the log-sum of every token
            s["dlse"] = 2e-4 * s["lse"] * s["dloss"] if case["weights"] == "weighted" else None
    elif case["op"].startswith("gated"):
        m, K, dt, counts = case["m"], case["K"], _DT[case["dtype"]], _counts(case, host)
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + c)
        rows = max(case["rows"], offsets[-1])
        s["counts"] = counts          # the host's copy: what the plain form cuts its products by
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        s["x"] = _normal((rows, K), 1.0, dt, gen)
        s["w"] = _normal((case["E"], 2 * m, K), K ** -0.5, dt, gen)
        if case["op"] == "gated_bwd":
            s["gu"] = _normal((rows, 2 * m), 1.0, dt, gen)      # what the forward left: unit normal, as x and w are
            s["dh"] = _normal((rows, m), 1.0, dt, gen)
            if rows > offsets[-1]:    # rows of no expert: whatever is there does not count
                s["x"][offsets[-1]:] = math.nan
                s["dh"][offsets[-1]:] = math.inf
                s["gu"][offsets[-1]:] = math.nan
    else:
        s["flats"], s["grads"] = [], []
        for kind, total, n in _flats(case):
            flat = _normal((total,), 1e-2, _DT[kind], gen)
            parts = list(flat.split(_lengths(total, n, host)))
            scales = torch.exp(torch.randn(n, generator=host)).tolist()
            for p, f in zip(parts, scales):     # parameters of different scales
                p.mul_(f)
            s["flats"].append(flat)
            s["grads"] += parts
        if case["op"] == "grad_clip":
            # a limit on either side of the norm
            norm = math.sqrt(sum(float(f.float().square().sum(dtype=torch.float64)) for f in s["flats"]))
            s["max_norm"] = case["limit"] * norm
            s["outs"] = s["out"] = None
            if case["place"] != "here":
                s["outs"] = [torch.empty(f.shape, dtype=torch.float32 if case["place"] == "masters" else f.dtype,
                                         device="cuda") for f in s["flats"]]
                sizes = [p.numel() for p in s["grads"]]
                s["out"] = []
                for o in s["outs"]:
                    n, at = len(s["out"]), 0
                    while at < o.numel():
                        s["out"].append(o[at:at + sizes[n]])
                        at, n = at + sizes[n], n + 1
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from mixture_experts_layer_device_gb300 import block
    c = s["case"]
    if c["op"] == "vocab_fwd":
        return block.vocab_loss_forward(s["x"], s["w"], s["labels"])
    if c["op"] == "vocab_bwd":
        return block.vocab_loss_backward(s["dloss"], s["x"], s["w"], s["labels"], s["lse"], dlse=s["dlse"])
    if c["op"] == "gated_fwd":
        return block.gated_forward(s["x"], s["w"], s["offsets"], act=c["act"], need_gu=c["save"])
    if c["op"] == "gated_bwd":
        return block.gated_backward(s["dh"], s["x"], s["w"], s["offsets"], s["gu"], act=c["act"])
    if c["op"] == "grad_norm":
        return block.grad_norm(s["grads"])
    norm = block.grad_clip(s["grads"], s["max_norm"], out=s["out"], eps=_EPS)
    return [norm] + (s["outs"] or s["flats"])


def _run_plain(s):
    op = s["case"]["op"]
    return {"vocab_fwd": _plain_vocab_fwd, "vocab_bwd": _plain_vocab_bwd, "gated_fwd": _plain_gated_fwd,
            "gated_bwd": _plain_gated_bwd, "grad_norm": _plain_grad_norm, "grad_clip": _plain_grad_clip}[op](s)


def _plain_vocab_fwd(s):
    x, w, labels = s["x"], s["w"], s["labels"]
    loss = torch.zeros(x.shape[0], dtype=torch.float32, device=x.device)
    lse = torch.zeros_like(loss)
    keep = torch.nonzero((labels >= 0) & (labels < w.shape[0]))[:, 0]
    z = x[keep].float() @ w.float().T
    most = z.max(1).values
    lse[keep] = most + torch.log(torch.exp(z - most[:, None]).sum(1))
    loss[keep] = lse[keep] - z.gather(1, labels[keep].long()[:, None])[:, 0]
    return loss, lse


def _plain_vocab_bwd(s):
    x, w, labels = s["x"], s["w"], s["labels"]
    dx = torch.zeros_like(x)
    keep = torch.nonzero((labels >= 0) & (labels < w.shape[0]))[:, 0]
    xf, wf, dloss = x[keep].float(), w.float(), s["dloss"][keep]
    both = dloss if s["dlse"] is None else dloss + s["dlse"][keep]
    dz = xf @ wf.T
    dz = torch.exp(dz - s["lse"][keep][:, None]) * both[:, None]
    dz[torch.arange(keep.numel(), device=x.device), labels[keep].long()] -= dloss
    dx[keep] = (dz @ wf).to(x.dtype)
    return dx, (dz.T @ xf).to(w.dtype)


def _act(kind, g, derivative=False):
    """act(g), or its derivative, in g's type."""
    if kind == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return sig * (1.0 + g * (1.0 - sig)) if derivative else g * sig
    if kind == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return cdf + g * torch.exp(-0.5 * g * g) * (0.5 / math.pi) ** 0.5 if derivative else g * cdf
    if kind == "gelu_tanh":
        a, b = math.sqrt(2.0 / math.pi), 0.044715
        t = torch.tanh(a * (g + b * g * g * g))
        if derivative:
            return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * a * (1.0 + 3.0 * b * g * g)
        return 0.5 * g * (1.0 + t)
    return (g > 0).to(g.dtype) if derivative else torch.where(g > 0, g, 0.0)


def _cut(s):
    """How the plain form takes the experts that have rows: as one batch padded
    to the largest load where that adds at most as many rows again, else one
    product for each, which is then the faster."""
    counts = s["counts"]
    active = [e for e, n in enumerate(counts) if n]
    most = max((counts[e] for e in active), default=0)
    return active, most, most * len(active) <= 2 * sum(counts)


def _slots(s, active, most):
    """Row of every place of the batch [active, most], and whether it has one."""
    dev = s["offsets"].device
    at = torch.tensor(active, device=dev)
    first, last = s["offsets"][at].long(), s["offsets"][at + 1].long()
    row = first[:, None] + torch.arange(most, device=dev)
    return at, row.clamp(max=s["x"].shape[0] - 1), row < last[:, None]


def _plain_gated_fwd(s):
    x, w, m, act = s["x"], s["w"], s["case"]["m"], s["case"]["act"]
    gu = torch.zeros((x.shape[0], 2 * m), dtype=x.dtype, device=x.device)
    h = torch.zeros((x.shape[0], m), dtype=x.dtype, device=x.device)
    active, most, batch = _cut(s)
    if batch:
        at, row, has = _slots(s, active, most)
        y = torch.matmul(x[row].float(), w[at].float().transpose(1, 2))[has]
        gu[row[has]] = y.to(x.dtype)
        h[row[has]] = (_act(act, y[:, :m]) * y[:, m:]).to(x.dtype)
        return h, gu if s["case"]["save"] else None
    r = 0
    for e, n in enumerate(s["counts"]):
        if n:
            y = x[r:r + n].float() @ w[e].float().T
            gu[r:r + n] = y.to(x.dtype)
            h[r:r + n] = (_act(act, y[:, :m]) * y[:, m:]).to(x.dtype)
        r += n
    return h, gu if s["case"]["save"] else None


def _plain_gated_bwd(s):
    x, w, m, act = s["x"], s["w"], s["case"]["m"], s["case"]["act"]
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    dh, g, u = s["dh"].float(), s["gu"][:, :m].float(), s["gu"][:, m:].float()
    dgu = torch.cat([dh * u * _act(act, g, True), dh * _act(act, g)], 1)
    active, most, batch = _cut(s)
    if batch:
        at, row, has = _slots(s, active, most)
        d = torch.where(has[..., None], dgu[row], 0.0)
        dx[row[has]] = torch.matmul(d, w[at].float())[has].to(dx.dtype)
        dw[at] = torch.matmul(d.transpose(1, 2), torch.where(has[..., None], x[row].float(), 0.0)).to(dw.dtype)
        return dx, dw
    r = 0
    for e, n in enumerate(s["counts"]):
        if n:
            d = dgu[r:r + n]
            dx[r:r + n] = (d @ w[e].float()).to(dx.dtype)
            dw[e] = (d.T @ x[r:r + n].float()).to(dw.dtype)
        r += n
    return dx, dw


def _plain_grad_norm(s):
    # 64 bits where the long sum ends: the squares of each gradient are added up in them
    return torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt().float()


def _plain_grad_clip(s):
    norm = _plain_grad_norm(s)
    c = torch.clamp(s["max_norm"] / (norm + _EPS), max=1.0)
    for g, o in zip(s["grads"], s["out"] or s["grads"]):
        o.copy_(g.float() * c)
    return [norm] + (s["outs"] or s["flats"])


# ---------------------------------------------------------------- exact values
def exact(case, seed):
    if work(case)["flops"] > 1.2e13:      # products in 64 bits run at about a TFLOP/s
        return None
    s = prepare(case, seed)
    d = torch.float64
    if case["op"].startswith("vocab"):
        x, w, T, V = s["x"], s["w"], case["rows"], case["V"]
        rows = [t for t, y in enumerate(s["labels"].tolist()) if 0 <= y < V]
        at = torch.tensor(rows, dtype=torch.long, device="cuda")
        xs, ys = x[at].to(d), s["labels"][at]
        if case["op"] == "vocab_fwd":
            loss, lse = torch.zeros(T, dtype=d, device="cuda"), torch.zeros(T, dtype=d, device="cuda")
            sums = torch.full((len(rows),), -math.inf, dtype=d, device="cuda")
            for lo in range(0, V, 16384):
                sums = torch.logaddexp(sums, torch.logsumexp(xs @ w[lo:lo + 16384].to(d).T, 1))
            lse[at] = sums
            loss[at] = sums - torch.einsum("td,td->t", xs, w[ys].to(d))
            return loss, lse
        a = s["dloss"][at].to(d)
        b = a if s["dlse"] is None else a + s["dlse"][at].to(d)
        dx = torch.zeros(x.shape, dtype=d, device="cuda")
        dw = torch.zeros(w.shape, dtype=d, device="cuda")
        part = torch.zeros(xs.shape, dtype=d, device="cuda")
        for lo in range(0, V, 16384):
            wp = w[lo:lo + 16384].to(d)
            dz = b[:, None] * torch.exp(xs @ wp.T - s["lse"][at].to(d)[:, None])
            here = torch.nonzero((ys >= lo) & (ys < lo + wp.shape[0]))[:, 0]
            dz[here, ys[here] - lo] -= a[here]
            part += dz @ wp
            dw[lo:lo + wp.shape[0]] = dz.T @ xs
        dx[at] = part
        return dx, dw
    if case["op"].startswith("gated"):
        ends, m, act = s["offsets"].tolist(), case["m"], case["act"]
        x, w = s["x"], s["w"]
        if case["op"] == "gated_fwd":
            gu = torch.zeros((x.shape[0], 2 * m), dtype=d, device="cuda")
            for e in range(case["E"]):
                lo, hi = ends[e], ends[e + 1]
                if hi > lo:
                    torch.matmul(x[lo:hi].to(d), w[e].to(d).T, out=gu[lo:hi])
            return _exact_act(act, gu[:, :m])[0] * gu[:, m:], gu if case["save"] else None
        dx = torch.zeros(x.shape, dtype=d, device="cuda")
        dw = torch.zeros(w.shape, dtype=d, device="cuda")
        for e in range(case["E"]):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                value, slope = _exact_act(act, s["gu"][lo:hi, :m].to(d))
                dh = s["dh"][lo:hi].to(d)
                dgu = torch.hstack((dh * s["gu"][lo:hi, m:].to(d) * slope, dh * value))
                torch.matmul(dgu, w[e].to(d), out=dx[lo:hi])
                torch.matmul(dgu.T, x[lo:hi].to(d), out=dw[e])
        return dx, dw
    norm = torch.zeros((), dtype=d, device="cuda")
    for f in s["flats"]:
        for piece in f.split(1 << 28):
            norm += torch.dot(piece.to(d), piece.to(d))
    norm = norm.sqrt()
    if case["op"] == "grad_norm":
        return norm
    c = min(1.0, s["max_norm"] / (float(norm) + _EPS))
    return [norm] + [f.to(d) * c for f in s["flats"]]


def _exact_act(kind, g):
    """(act(g), act'(g)) in 64 bits, written by other identities than the plain form's."""
    if kind == "silu":        # g / 2 (1 + tanh(g / 2))
        t = torch.tanh(0.5 * g)
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.25 * g * (1.0 - t * t)
    if kind == "gelu":        # g Phi(g) by the complementary error function
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":   # g sigmoid(2 a (g + b g^3))
        a, b = math.sqrt(2.0 / math.pi), 0.044715
        sig = torch.sigmoid(2.0 * a * (g + b * g ** 3))
        return g * sig, sig + g * sig * (1.0 - sig) * 2.0 * a * (1.0 + 3.0 * b * g ** 2)
    return g.clamp(min=0.0), torch.heaviside(g, torch.zeros((), dtype=g.dtype, device=g.device))


# ---------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass: every input that counts read once,
    every output written once."""
    if case["op"].startswith("vocab"):
        T, V, d, b = case["rows"], case["V"], case["d"], _BYTES[case["dtype"]]
        n = max(1, round(T * (1.0 - case["ignored"])))
        if case["op"] == "vocab_fwd":
            return dict(bytes=n * d * b + V * d * b + 8 * T + 8 * T, flops=2 * n * V * d)
        # without keeping the logits they are formed again
        return dict(bytes=n * d * b + V * d * b + 16 * T + T * d * b + V * d * b, flops=6 * n * V * d)
    if case["op"].startswith("gated"):
        rows, m, K, b = max(case["rows"], case["active"]), case["m"], case["K"], _BYTES[case["dtype"]]
        w, x, h = case["active"] * 2 * m * K * b, rows * K * b, rows * m * b
        if case["op"] == "gated_fwd":
            return dict(bytes=x + w + h + (2 * h if case["save"] else 0) + 4 * (case["E"] + 1), flops=4 * rows * m * K)
        return dict(bytes=3 * h + x + w + x + case["E"] * 2 * m * K * b + 4 * (case["E"] + 1), flops=8 * rows * m * K)
    read = sum(total * _BYTES[kind] for kind, total, _ in _flats(case))
    if case["op"] == "grad_norm":
        return dict(bytes=read, flops=2 * case["total"])
    # in place below the limit nothing has to be written
    written = {"masters": 4 * case["total"], "apart": read, "here": read if case["limit"] < 1.0 else 0}[case["place"]]
    return dict(bytes=read + written, flops=3 * case["total"])
