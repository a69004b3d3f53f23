"""Cases, plain forms and exact values of the operators around the MoE layer:
the ragged products grouped by expert, the norms around a block with its gate
and residual scale, and the token embedding with its gradient.

`run` computes a case in its plain form (elementary torch operations in fp32,
rounded once), or through this package's kernels where `own` is true; `exact`
gives the same outputs in 64 bits from the definitions.

  grouped    Y[r] = X[r] W[e]^T for the rows r of expert e (offsets[e] ..
             offsets[e+1]); dX[r] = dY[r] W[e]; dW[e] = sum_r dY[r]^T X[r];
             rows of no expert give 0
  norm       z = alpha x + g * (w_post * f / rms(f)), h = w_pre * z / rms(z),
             rms(v) = sqrt(mean(v^2) + eps); without the post norm f enters
             as it is; backward of all inputs and weights
  embed      out[t] = scale * table[ids[t]] (0 for an id outside the table),
             dtable[v] = scale * sum of dout[t] over the t with ids[t] = v
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
        # one generated token through the gate/up product of a layer with 512 experts, top 10 (the
        # layer's Qwen3.5-397B-A17B shape): ten rows, ten weight matrices
        dict(name="grouped_fwd_one_token", op="grouped_fwd", rows=10, E=512, active=10, N=2048, K=4096,
             spread=0.0, outside=0, dtype="bf16"),
        # low-rank adapters of odd sizes under a small serving batch; 7 experts get nothing
        dict(name="grouped_fwd_odd", op="grouped_fwd", rows=777, E=40, active=33, N=513, K=251,
             spread=0.7, outside=5, dtype="fp16"),
        # the gate/up product of a prompt or training step of the same layer: 8192 tokens, top 10
        dict(name="grouped_fwd_sequence", op="grouped_fwd", rows=81920, E=512, active=512, N=2048, K=4096,
             spread=0.3, outside=0, dtype="bf16"),
        # a training step's down-projection gradients with skewed loads and four idle experts
        dict(name="grouped_bwd_skewed", op="grouped_bwd", rows=32768, E=64, active=60, N=7168, K=2048,
             spread=1.2, outside=0, dtype="bf16"),
        # a small fine-tuning step
        dict(name="grouped_bwd_small", op="grouped_bwd", rows=2043, E=8, active=8, N=512, K=768,
             spread=0.5, outside=3, dtype="fp16"),
        # one generated token between two blocks (Kimi-K2.7 width)
        dict(name="norm_fwd_one_token", op="norm_fwd", rows=1, d=7168, gate="channel", post=True, pre=True,
             alpha=1.0, dtype="bf16"),
        # a prompt or training step of 16,384 tokens between two blocks, gated by token
        dict(name="norm_fwd_sequence", op="norm_fwd", rows=16384, d=7168, gate="row", post=True, pre=True,
             alpha=0.7, dtype="bf16"),
        # the backward of a training step (GLM-5.2 width), gated by channel
        dict(name="norm_bwd_sequence", op="norm_bwd", rows=16384, d=6144, gate="channel", post=True, pre=True,
             alpha=1.0, dtype="bf16"),
        # a ragged batch at an odd width, a gate for every element
        dict(name="norm_bwd_odd", op="norm_bwd", rows=1531, d=2883, gate="full", post=True, pre=True,
             alpha=0.5, dtype="fp16"),
        # a training step's lookup
        dict(name="embed_fwd_sequence", op="embed_fwd", rows=16384, V=131072, d=4096, pad=0.0, ids="int64",
             dtype="bf16"),
        # the dense gradient of a training step's table; token frequencies fall as 1 / rank
        dict(name="embed_bwd_sequence", op="embed_bwd", rows=32768, V=131072, d=4096, pad=0.03, ids="int64",
             dtype="bf16"),
        # the table of a small model at odd sizes, fp32
        dict(name="embed_bwd_odd", op="embed_bwd", rows=515, V=50001, d=321, pad=0.1, ids="int32",
             dtype="fp32"),
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
    n = min(n, hi)
    return n + 64 if n == 3072 else n


def draw(rng):
    op = rng.choice(["grouped_fwd", "grouped_bwd", "norm_fwd", "norm_bwd", "embed_fwd", "embed_bwd"])
    if op.startswith("grouped"):
        most = {"grouped_fwd": 81920 * 2048 * 4096, "grouped_bwd": 32768 * 7168 * 2048}[op]
        while True:
            E = _log(rng, 1, 512)
            c = dict(op=op, rows=_log(rng, 1, 81920), E=E, active=0, N=_size(rng, 16, 7168), K=_size(rng, 16, 7168),
                     spread=rng.choice([0.0, 0.4, 1.0]), outside=rng.choice([0, 0, 3]),
                     dtype=rng.choice(["bf16", "bf16", "fp16"]))
            c["active"] = min(c["rows"], max(1, round(E * rng.uniform(0.5, 1.0))))
            if c["rows"] * c["N"] * c["K"] <= most and c["active"] * c["N"] * c["K"] <= most // 160:
                return c
    if op.startswith("norm"):
        while True:
            c = dict(op=op, rows=_log(rng, 1, 65536), d=_size(rng, 64, 16384),
                     gate=rng.choice(["none", "channel", "row", "full"]), post=rng.random() < 0.7,
                     pre=rng.random() < 0.8, alpha=rng.choice([1.0, 0.5]),
                     dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
            c["pre"] = c["pre"] or not c["post"]
            if c["rows"] * c["d"] * (_BYTES[c["dtype"]] + (2 if c["gate"] == "full" else 0)) <= 16384 * 6144 * 2:
                return c
    while True:
        c = dict(op=op, rows=_log(rng, 1, 65536), V=_log(rng, 100, 131072), d=_size(rng, 16, 8192),
                 pad=rng.choice([0.0, 0.1]), ids=rng.choice(["int64", "int32"]),
                 dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
        most = 16384 * 4096 * 2 if op == "embed_fwd" else 32768 * 4096 * 2
        if c["rows"] * c["d"] * _BYTES[c["dtype"]] <= most and c["V"] * c["d"] * _BYTES[c["dtype"]] <= 131072 * 4096 * 2:
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


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    s = dict(case=dict(case))
    if case["op"].startswith("grouped"):
        N, K, counts = case["N"], case["K"], _counts(case, host)
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + c)
        rows = max(case["rows"], offsets[-1])
        s["counts"] = counts          # the host's copy: what the plain form cuts its products by
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        s["x"] = _normal((rows, K), 1.0, dt, gen)
        s["w"] = _normal((case["E"], N, K), K ** -0.5, dt, gen)
        if case["op"] == "grouped_bwd":
            s["dy"] = _normal((rows, N), 1.0, dt, gen)
            if rows > offsets[-1]:    # rows of no expert: whatever is there does not count
                s["x"][offsets[-1]:] = math.nan
                s["dy"][offsets[-1]:] = math.inf
    elif case["op"].startswith("norm"):
        T, d = case["rows"], case["d"]
        s["x"] = _normal((T, d), 1.0, dt, gen)
        # a block's output: rows of different scales, a few channels that stand out
        f = torch.randn((T, d), generator=gen, device="cuda")
        f *= torch.exp(0.7 * torch.randn((T, 1), generator=gen, device="cuda"))
        f[:, ::97] *= 4.0
        s["f"] = f.to(dt)
        one = lambda *n: (1.0 + 0.2 * torch.randn(n, generator=gen, device="cuda")).to(dt)  # noqa: E731
        s["w_post"] = one(d) if case["post"] else None
        s["w_pre"] = one(d) if case["pre"] else None
        shape = {"none": None, "channel": (d,), "row": (T,), "full": (T, d)}[case["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(torch.randn(shape, generator=gen, device="cuda")).to(dt)
        if case["op"] == "norm_bwd":
            # what the forward left: the summed residual and the reciprocal roots, and the gradients that arrive
            f, r_post = s["f"].float(), None
            n = f
            if case["post"]:
                r_post = torch.rsqrt(f.square().mean(1) + _EPS)
                n = f * r_post[:, None] * s["w_post"].float()
            gate = s["gate"].float() if s["gate"] is not None else torch.ones((), device="cuda")
            z = case["alpha"] * s["x"].float() + (gate[:, None] if case["gate"] == "row" else gate) * n
            s["z"], s["r_post"] = z.to(dt), r_post
            s["r_pre"] = torch.rsqrt(z.square().mean(1) + _EPS) if case["pre"] else None
            s["dz"] = _normal((T, d), 1.0, dt, gen)
            s["dh"] = _normal((T, d), 1.0, dt, gen) if case["pre"] else None
            del s["x"]
    else:
        T, V, d = case["rows"], case["V"], case["d"]
        # token frequencies fall as 1 / rank, ranks spread over the table; padding is -1
        u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64)
        rank = torch.exp(u * math.log(V)).long().clamp_(1, V) - 1
        ids = torch.randperm(V, generator=gen, device="cuda")[rank]
        ids[torch.rand(T, generator=gen, device="cuda") < case["pad"]] = -1
        s["ids"] = ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)
        s["scale"] = float(d) ** 0.5 if case["op"] == "embed_fwd" else 0.5
        if case["op"] == "embed_fwd":
            s["table"] = _normal((V, d), 0.02, dt, gen)
        else:
            s["dout"] = _normal((T, d), 1.0, dt, gen)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from mixture_experts_layer_device_gb300 import block
    c = s["case"]
    if c["op"] == "grouped_fwd":
        return block.grouped_forward(s["x"], s["w"], s["offsets"])
    if c["op"] == "grouped_bwd":
        return block.grouped_backward(s["dy"], s["x"], s["w"], s["offsets"])
    if c["op"] == "norm_fwd":
        return block.norm_forward(s["x"], s["f"], s["gate"], s["w_post"], s["w_pre"], gate_kind=c["gate"],
                                  post=c["post"], pre=c["pre"], alpha=c["alpha"], eps=_EPS)
    if c["op"] == "norm_bwd":
        return block.norm_backward(s["dz"], s["dh"], s["z"], s["f"], s["gate"], s["w_post"], s["w_pre"], s["r_post"],
                                   s["r_pre"], gate_kind=c["gate"], post=c["post"], pre=c["pre"], alpha=c["alpha"])
    if c["op"] == "embed_fwd":
        return block.embed_forward(s["ids"], s["table"], scale=s["scale"])
    return block.embed_backward(s["ids"], s["dout"], c["V"], scale=s["scale"])


def _run_plain(s):
    op = s["case"]["op"]
    return {"grouped_fwd": _plain_grouped_fwd, "grouped_bwd": _plain_grouped_bwd, "norm_fwd": _plain_norm_fwd,
            "norm_bwd": _plain_norm_bwd, "embed_fwd": _plain_embed_fwd, "embed_bwd": _plain_embed_bwd}[op](s)


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


def _plain_grouped_fwd(s):
    x, w = s["x"], s["w"]
    y = torch.zeros((x.shape[0], w.shape[1]), dtype=x.dtype, device=x.device)
    active, most, batch = _cut(s)
    if batch:
        at, row, has = _slots(s, active, most)
        y[row[has]] = torch.matmul(x[row].float(), w[at].float().transpose(1, 2))[has].to(y.dtype)
        return y
    r = 0
    for e, n in enumerate(s["counts"]):
        if n:
            y[r:r + n] = (x[r:r + n].float() @ w[e].float().T).to(y.dtype)
        r += n
    return y


def _plain_grouped_bwd(s):
    dy, x, w = s["dy"], s["x"], s["w"]
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    active, most, batch = _cut(s)
    if batch:
        at, row, has = _slots(s, active, most)
        g = torch.where(has[..., None], dy[row].float(), 0.0)
        dx[row[has]] = torch.matmul(g, w[at].float())[has].to(dx.dtype)
        dw[at] = torch.matmul(g.transpose(1, 2), torch.where(has[..., None], x[row].float(), 0.0)).to(dw.dtype)
        return dx, dw
    r = 0
    for e, n in enumerate(s["counts"]):
        if n:
            g = dy[r:r + n].float()
            dx[r:r + n] = (g @ w[e].float()).to(dx.dtype)
            dw[e] = (g.T @ x[r:r + n].float()).to(dw.dtype)
        r += n
    return dx, dw


def _gate(s, like):
    g = s["gate"]
    if g is None:
        return torch.ones((), dtype=like, device=s["f"].device)
    g = g.to(like)
    return g[:, None] if s["case"]["gate"] == "row" else g


def _plain_norm_fwd(s):
    c, dt = s["case"], s["x"].dtype
    n, r_post, h, r_pre = s["f"].float(), None, None, None
    if c["post"]:
        r_post = torch.rsqrt(n.square().mean(1) + _EPS)
        n = n * r_post[:, None] * s["w_post"].float()
    z = c["alpha"] * s["x"].float() + _gate(s, torch.float32) * n
    if c["pre"]:
        r_pre = torch.rsqrt(z.square().mean(1) + _EPS)
        h = (z * r_pre[:, None] * s["w_pre"].float()).to(dt)
    return z.to(dt), h, r_post, r_pre


def _plain_norm_bwd(s):
    c, dt, kind = s["case"], s["dz"].dtype, s["case"]["gate"]
    dz, f, gate = s["dz"].float(), s["f"].float(), _gate(s, torch.float32)
    dw_pre = dw_post = dgate = None
    if c["pre"]:
        dh, r = s["dh"].float(), s["r_pre"][:, None]
        zn = s["z"].float() * r
        dw_pre = (dh * zn).sum(0).to(dt)
        dn = dh * s["w_pre"].float()
        dz = dz + r * (dn - zn * (dn * zn).mean(1, keepdim=True))
    fn = f * s["r_post"][:, None] if c["post"] else f
    n = fn * s["w_post"].float() if c["post"] else fn
    if kind != "none":
        dgate = dz * n
        dgate = (dgate.sum(0) if kind == "channel" else dgate.sum(1) if kind == "row" else dgate).to(dt)
    df = dz * gate
    if c["post"]:
        dw_post = (df * fn).sum(0).to(dt)
        df = df * s["w_post"].float()
        df = s["r_post"][:, None] * (df - fn * (df * fn).mean(1, keepdim=True))
    return (c["alpha"] * dz).to(dt), df.to(dt), dgate, dw_post, dw_pre


def _plain_embed_fwd(s):
    ids, table = s["ids"].long(), s["table"]
    ok = (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(ok, ids, 0)].float() * s["scale"]
    return torch.where(ok[:, None], rows, 0.0).to(table.dtype)


def _plain_embed_bwd(s):
    V, ids, dout = s["case"]["V"], s["ids"].long(), s["dout"]
    ok = (ids >= 0) & (ids < V)
    total = torch.zeros((V + 1, dout.shape[1]), dtype=torch.float32, device=dout.device)
    total.index_add_(0, torch.where(ok, ids, V), dout.float())
    return (total[:V] * s["scale"]).to(dout.dtype)


# ---------------------------------------------------------------- exact values
def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"].startswith("grouped"):
        ends = s["offsets"].tolist()
        x, w = s["x"], s["w"]
        if case["op"] == "grouped_fwd":
            y = torch.zeros((x.shape[0], w.shape[1]), dtype=d, device="cuda")
            for e in range(case["E"]):
                lo, hi = ends[e], ends[e + 1]
                if hi > lo:
                    torch.matmul(x[lo:hi].to(d), w[e].to(d).T, out=y[lo:hi])
            return y
        dx = torch.zeros(x.shape, dtype=d, device="cuda")
        dw = torch.zeros(w.shape, dtype=d, device="cuda")
        for e in range(case["E"]):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                g = s["dy"][lo:hi].to(d)
                torch.matmul(g, w[e].to(d), out=dx[lo:hi])
                torch.matmul(g.T, x[lo:hi].to(d), out=dw[e])
        return dx, dw
    if case["op"].startswith("norm"):
        f, gate = s["f"].to(d), _gate(s, d)
        w_post = s["w_post"].to(d) if case["post"] else None
        if case["op"] == "norm_fwd":
            r_post = (f.pow(2).mean(1) + _EPS).pow(-0.5) if case["post"] else None
            z = case["alpha"] * s["x"].to(d)
            z += gate * (f * (r_post[:, None] * w_post) if case["post"] else f)
            if not case["pre"]:
                return z, None, r_post, None
            r_pre = (z.pow(2).mean(1) + _EPS).pow(-0.5)
            return z, z * r_pre[:, None] * s["w_pre"].to(d), r_post, r_pre
        # u = r v, r = (mean v^2 + eps)^-1/2:  du -> dv = r du - v r^3 <du, v> / d
        dz, width, dw_pre, dw_post, dgate = s["dz"].to(d), case["d"], None, None, None
        if case["pre"]:
            z, r, dh = s["z"].to(d), s["r_pre"].to(d)[:, None], s["dh"].to(d)
            dw_pre = torch.einsum("td,td->d", dh, z * r)
            du = dh * s["w_pre"].to(d)
            dz = dz + r * du - z * (r.pow(3) * (du * z).sum(1, keepdim=True) / width)
        r = s["r_post"].to(d)[:, None] if case["post"] else None
        n = f * r * w_post if case["post"] else f
        if case["gate"] == "channel":
            dgate = torch.einsum("td,td->d", dz, n)
        elif case["gate"] == "row":
            dgate = torch.einsum("td,td->t", dz, n)
        elif case["gate"] == "full":
            dgate = dz * n
        df = dz * gate
        if case["post"]:
            dw_post = torch.einsum("td,td->d", df, f * r)
            du = df * w_post
            df = r * du - f * (r.pow(3) * (du * f).sum(1, keepdim=True) / width)
        return case["alpha"] * dz, df, dgate, dw_post, dw_pre
    ids = s["ids"].long()
    if case["op"] == "embed_fwd":
        out = torch.zeros((case["rows"], case["d"]), dtype=d, device="cuda")
        has = torch.nonzero((ids >= 0) & (ids < case["V"]))[:, 0]
        out[has] = s["table"][ids[has]].to(d) * s["scale"]
        return out
    has = torch.nonzero((ids >= 0) & (ids < case["V"]))[:, 0]
    out = torch.zeros((case["V"], case["d"]), dtype=d, device="cuda")
    out.index_add_(0, ids[has], s["dout"][has].to(d) * s["scale"])
    return out


# ---------------------------------------------------------------- work
def work(case):
    """Bytes and operations of one pass: every input that counts read once,
    every output written once."""
    b = _BYTES[case["dtype"]]
    if case["op"].startswith("grouped"):
        rows, N, K = max(case["rows"], case["active"]), case["N"], case["K"]
        w, x, y = case["active"] * N * K * b, rows * K * b, rows * N * b
        if case["op"] == "grouped_fwd":
            return dict(bytes=x + w + y + 4 * (case["E"] + 1), flops=2 * rows * N * K)
        return dict(bytes=y + x + w + x + case["E"] * N * K * b + 4 * (case["E"] + 1), flops=4 * rows * N * K)
    if case["op"].startswith("norm"):
        T, d = case["rows"], case["d"]
        gate = {"none": 0, "channel": d, "row": T, "full": T * d}[case["gate"]] * b
        weights = (case["post"] + case["pre"]) * d * b
        roots = 4 * T * (case["post"] + case["pre"])
        if case["op"] == "norm_fwd":   # f, x in; z, h out
            return dict(bytes=T * d * b * (3 + case["pre"]) + gate + weights + roots, flops=10 * T * d)
        # dz, f in (with the pre norm dh, z too); dx, df out
        return dict(bytes=T * d * b * (4 + 2 * case["pre"]) + 2 * gate + 2 * weights + roots, flops=20 * T * d)
    T, V, d = case["rows"], case["V"], case["d"]
    ids = T * (4 if case["ids"] == "int32" else 8)
    if case["op"] == "embed_fwd":
        return dict(bytes=2 * T * d * b + ids, flops=T * d)
    return dict(bytes=T * d * b + V * d * b + ids, flops=T * d)
