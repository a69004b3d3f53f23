"""A torch drop-in for the MoE layer: an autograd.Function around the C ABI
and an nn.Module that owns the bf16 master weights as parameters.

Every computation runs in the library's kernels; this file only moves
pointers.  The forward re-derives the kernels' weight operands (MXFP8 codes in
both orientations, or bf16 transposes) from the current masters, so an
optimizer step on the parameters is seen by the next forward; its cost is the
weight preparation step of a training update.  Gradients pass straight through
the MXFP8 quantisers, so the masters receive the gradients the library
computes for the quantised layer.  Each training forward keeps its activations
in its own buffer, so several forwards may precede their backwards.

Around the layer: GroupedLinear (ragged products grouped by expert),
GatedLinear (the same with a gate and its activation), BlockNorm (the norms
around a block with its gate and residual scale), TokenEmbedding and VocabLoss
(the loss over a vocabulary without its logits), each an nn.Module over an
autograd.Function over block.py; clip_gradients for all of them.

Gradients have no second derivative: under create_graph they refuse one.
"""
import torch

from . import block
from .layer import MoELayer


class _FirstOrder(torch.autograd.Function):
    """A gradient as it is, which cannot be differentiated."""

    @staticmethod
    def forward(ctx, grad, *depends):
        return grad

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the second derivative of the library's operators is not built: this gradient was computed "
                           "under create_graph and is differentiated")


def _first_order(grad, *depends):
    """`grad`, computed out of autograd's sight from `depends`.  Where a graph is asked
    for (create_graph), it refuses to be differentiated instead of passing for a
    constant."""
    if grad is None or not torch.is_grad_enabled() or not any(t is not None and t.requires_grad for t in depends):
        return grad
    return _FirstOrder.apply(grad, *depends)


class MoEFunction(torch.autograd.Function):
    """y = moe(x, logits; W_gu, W_dn[, Ws_gu, Ws_dn]) for the shapes of `layer`.

    x [T, d] bf16, logits [T, E] fp32 -> y [T, d] bf16.  With router weights
    W_r [E, d] (bf16) the logits are computed from x instead (pass logits =
    None); the router's backward then adds its dx contribution in place and
    returns dW_r.  Backward returns dx, dlogits (fp32; with a load-balancing
    term its gradient is included) and the gradients of the bf16 weights."""

    @staticmethod
    def forward(ctx, x, logits, W_r, W_gu, W_dn, Ws_gu, Ws_dn, layer):
        layer.prepare_from(W_gu, W_dn, Ws_gu, Ws_dn)
        x = x.contiguous()
        if W_r is not None:
            logits = layer.router_logits(x, W_r.contiguous())
        need = any(ctx.needs_input_grad[:7])
        saved = layer.new_saved() if need else None
        y = layer.forward(x, logits.contiguous(), train=need, saved=saved)
        if need:
            ctx.layer, ctx.saved, ctx.router = layer, saved, W_r is not None
            ctx.save_for_backward(x, W_r if W_r is not None else x)
        return y

    @staticmethod
    def backward(ctx, dy):
        # The backward reads the weight operands of the current masters: they
        # must not change between a forward and its backward (no optimizer
        # step in between), as in every usual training schedule.
        x, W_r = ctx.saved_tensors
        layer = ctx.layer
        g = layer.backward(dy.contiguous(), x, saved=ctx.saved)
        ctx.saved = None
        dW_r = None
        if ctx.router:
            dW_r = torch.empty_like(W_r)
            layer.router_backward(g["dlogits"], x, W_r.contiguous(), g["dx"], dW_r)
        grads = (g["dx"], None if ctx.router else g["dlogits"], dW_r, g["dW_gu"], g["dW_dn"], g["dWs_gu"], g["dWs_dn"])
        if torch.is_grad_enabled():     # every gradient depends on every input; the weights are not saved
            some = torch.zeros((), device=x.device, requires_grad=True)
            grads = tuple(_first_order(t, some) for t in grads)
        return grads + (None,)


class MoE(torch.nn.Module):
    """MoE layer for T tokens per call: E experts (gate/up [2m, d] and down
    [d, m] each, bf16 masters), top-k routing, optional BF16 shared expert of
    intermediate m_shared; fmt "mxfp8" or "bf16" for the routed experts.
    router=True adds router weights W_r [E, d] (forward(x)); otherwise the
    logits are given (forward(x, logits)).  aux_alpha > 0 adds the
    load-balancing term: its value after a forward is `aux_loss()` (a device
    scalar) and its gradient is applied inside the backward with weight 1, so
    it is not added to the loss again.  ring_rows / gather_sms select the
    dispatch ring (MXFP8)."""

    def __init__(self, T, d, m, E, k, fmt="mxfp8", m_shared=0, device="cuda", ring_rows=0, gather_sms=0,
                 router=False, aux_alpha=0.0):
        super().__init__()
        bf = dict(dtype=torch.bfloat16, device=device)
        self.W_r = torch.nn.Parameter(torch.empty(E, d, **bf).normal_(0.0, d ** -0.5)) if router else None
        self.W_gu = torch.nn.Parameter(torch.empty(E, 2 * m, d, **bf).normal_(0.0, d ** -0.5))
        self.W_dn = torch.nn.Parameter(torch.empty(E, d, m, **bf).normal_(0.0, m ** -0.5))
        if m_shared:
            self.Ws_gu = torch.nn.Parameter(torch.empty(2 * m_shared, d, **bf).normal_(0.0, d ** -0.5))
            self.Ws_dn = torch.nn.Parameter(torch.empty(d, m_shared, **bf).normal_(0.0, m_shared ** -0.5))
        else:
            self.Ws_gu = self.Ws_dn = None
        with torch.no_grad():
            shared = (self.Ws_gu, self.Ws_dn) if m_shared else None
            self.layer = MoELayer(T, d, m, E, k, fmt, shared=shared, backward=True, device=device,
                                  stacked=(self.W_gu, self.W_dn), ring_rows=ring_rows, gather_sms=gather_sms,
                                  aux_alpha=aux_alpha)

    def forward(self, x, logits=None):
        if (logits is None) != (self.W_r is not None):
            raise ValueError("pass logits exactly when the module has no router")
        return MoEFunction.apply(x, logits, self.W_r, self.W_gu, self.W_dn, self.Ws_gu, self.Ws_dn, self.layer)

    def aux_loss(self):
        """The load-balancing loss of the last forward (0-d fp32 device tensor)."""
        return self.layer.view(1, "aux", "f32", (1,))[0]


# ---------------------------------------------------------------- around the layer
class GroupedFunction(torch.autograd.Function):
    """y[r] = x[r] w[e]^T for the rows r of expert e (block.grouped_forward)."""

    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return block.grouped_forward(x, w, offsets)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[:2]
        dx = dw = None
        if need_dx or need_dw:
            dx, dw = block.grouped_backward(dy, x, w, offsets, need_dx=need_dx, need_dw=need_dw)
        return _first_order(dx, dy, w), _first_order(dw, dy, x), None


class GroupedLinear(torch.nn.Module):
    """E bias-free linear maps K -> N over expert-sorted rows: forward(x [rows, K],
    offsets int32 [E + 1]) -> [rows, N]; rows outside the offsets give zeros and
    take no gradient.  Weight [E, N, K] bf16 (or fp16)."""

    def __init__(self, E, N, K, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(E, N, K, dtype=dtype, device=device).normal_(0.0, K ** -0.5))

    def forward(self, x, offsets):
        return GroupedFunction.apply(x, self.weight, offsets)


class GatedFunction(torch.autograd.Function):
    """h[r] = act(x[r] w[e][:m]^T) (x[r] w[e][m:]^T) for the rows r of expert e (block.gated_forward)."""

    @staticmethod
    def forward(ctx, x, w, offsets, act):
        h, gu = block.gated_forward(x, w, offsets, act=act, need_gu=any(ctx.needs_input_grad[:2]))
        ctx.act = act
        ctx.save_for_backward(x, w, offsets, gu)
        return h

    @staticmethod
    def backward(ctx, dh):
        x, w, offsets, gu = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[:2]
        dx = dw = None
        if need_dx or need_dw:
            dx, dw = block.gated_backward(dh, x, w, offsets, gu, act=ctx.act, need_dx=need_dx, need_dw=need_dw)
        return _first_order(dx, dh, x, w), _first_order(dw, dh, x, w), None, None


class GatedLinear(torch.nn.Module):
    """The first half of E gated feed-forward blocks K -> m over expert-sorted rows:
    forward(x [rows, K], offsets int32 [E + 1]) -> act(x W_g^T) (x W_u^T) [rows, m]; rows
    outside the offsets give zeros and take no gradient.  Weight [E, 2m, K] bf16 (or
    fp16), an expert's W_g above its W_u; act "silu", "gelu", "gelu_tanh" or "relu".  A
    GroupedLinear(E, N, m) behind it makes the block whole."""

    def __init__(self, E, m, K, act="silu", dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(E, 2 * m, K, dtype=dtype, device=device).normal_(0.0, K ** -0.5))
        self.act = act

    def forward(self, x, offsets):
        if not torch.is_grad_enabled():     # a Function does not see the grad mode: it would write g and u
            return block.gated_forward(x, self.weight, offsets, act=self.act, need_gu=False)[0]
        return GatedFunction.apply(x, self.weight, offsets, self.act)


class BlockNormFunction(torch.autograd.Function):
    """(z, h) of block.norm_forward; z is None without need_z, h without pre."""

    @staticmethod
    def forward(ctx, x, f, gate, w_post, w_pre, gate_kind, post, pre, alpha, eps):
        post, alpha = post and f is not None, float(alpha)
        z, h, r_post, r_pre = block.norm_forward(x, f, gate, w_post, w_pre, gate_kind=gate_kind, post=post, pre=pre,
                                                 alpha=alpha, eps=eps)
        ctx.opts = dict(gate_kind=gate_kind, post=post, pre=pre, alpha=alpha)
        ctx.save_for_backward(z if pre else None, f, gate, w_post, w_pre, r_post, r_pre)
        ctx.set_materialize_grads(False)
        return z, h

    @staticmethod
    def backward(ctx, dz, dh):
        z, f, gate, w_post, w_pre, r_post, r_pre = ctx.saved_tensors
        need, opts = ctx.needs_input_grad, dict(ctx.opts)
        if dz is None and dh is None:
            return (None,) * 10
        if dh is None and opts["pre"]:      # only z was used: the pre norm has no part in it
            opts["pre"], z, r_pre = False, None, None
        dx, df, dgate, dw_post, dw_pre = block.norm_backward(
            dz, dh, z, f, gate, w_post, w_pre if opts["pre"] else None, r_post, r_pre, need_dx=need[0], need_df=need[1],
            need_dgate=need[2], need_dw=need[3] or need[4], **opts)
        grads = (dx, df, dgate, dw_post if need[3] else None, dw_pre if need[4] else None)
        return tuple(_first_order(t, dz, dh, z, f, gate, w_post, w_pre) for t in grads) + (None,) * 5


class BlockNorm(torch.nn.Module):
    """What stands between two blocks, in one pass over the tokens:

        z = alpha x + g * (w_post * f / rms(f)),   h = w_pre * z / rms(z)

    forward(x, f=None, gate=None) -> (z, h): x [T, d] the residual stream, f [T,
    d] the block's output (None: z = alpha x), h the next block's input.  post
    and pre leave the norms in; gate "none", "channel" (a parameter [d], ones at
    the start), "row" or "full" (given to forward, [T] or [T, d])."""

    def __init__(self, d, post=True, pre=True, gate="none", alpha=1.0, eps=1e-6, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        ones = lambda on: torch.nn.Parameter(torch.ones(d, dtype=dtype, device=device)) if on else None  # noqa: E731
        self.w_post, self.w_pre, self.w_gate = ones(post), ones(pre), ones(gate == "channel")
        self.post, self.pre, self.gate, self.alpha, self.eps = post, pre, gate, alpha, eps

    def forward(self, x, f=None, gate=None):
        kind = self.gate if f is not None else "none"
        if (gate is not None) != (kind in ("row", "full")):
            raise ValueError("pass a gate exactly when the module's kind is row or full and f is given")
        if kind == "channel":
            gate = self.w_gate
        return BlockNormFunction.apply(x, f, gate, self.w_post if f is not None else None, self.w_pre, kind, self.post,
                                       self.pre, self.alpha, self.eps)


class EmbeddingFunction(torch.autograd.Function):
    """scale * table[ids] (block.embed_forward), its gradient by sorted tokens."""

    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.V, ctx.scale = table.shape[0], float(scale)
        return block.embed_forward(ids, table, scale=ctx.scale)

    @staticmethod
    def backward(ctx, dout):
        ids, = ctx.saved_tensors
        return None, _first_order(block.embed_backward(ids, dout, ctx.V, scale=ctx.scale), dout), None


class TokenEmbedding(torch.nn.Module):
    """forward(ids) = scale * weight[ids]; an id outside [0, V) (padding) gives zeros
    and takes no gradient.  Weight [V, d]; the gradient is dense."""

    def __init__(self, V, d, scale=1.0, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(V, d, dtype=dtype, device=device).normal_(0.0, 0.02))
        self.scale = scale

    def forward(self, ids):
        return EmbeddingFunction.apply(ids, self.weight, self.scale)


class VocabLossFunction(torch.autograd.Function):
    """(loss, lse) of every row (block.vocab_loss_forward)."""

    @staticmethod
    def forward(ctx, x, w, labels):
        loss, lse = block.vocab_loss_forward(x, w, labels)
        ctx.save_for_backward(x, w, labels, lse)
        ctx.set_materialize_grads(False)
        return loss, lse

    @staticmethod
    def backward(ctx, dloss, dlse):
        x, w, labels, lse = ctx.saved_tensors
        need_dx, need_dw = ctx.needs_input_grad[:2]
        dx = dw = None
        if (need_dx or need_dw) and not (dloss is None and dlse is None):
            dx, dw = block.vocab_loss_backward(dloss, x, w, labels, lse, dlse=dlse, need_dx=need_dx, need_dw=need_dw)
        return _first_order(dx, dloss, dlse, x, w), _first_order(dw, dloss, dlse, x, w), None


class VocabLoss(torch.nn.Module):
    """Softmax cross entropy straight from the last hidden rows: forward(x [T, d],
    labels [T]) -> (loss [T], lse [T]) fp32, the logits x W^T never in memory.  A row
    whose label lies outside [0, V) (padding) gives zeros and takes no gradient; the
    mean over the others is loss.sum() / their number.  lse is there for a term in the
    logits' size (lse.square()).  Weight [V, d], or the given one (a TokenEmbedding's)."""

    def __init__(self, V, d, weight=None, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        if weight is None:
            weight = torch.nn.Parameter(torch.empty(V, d, dtype=dtype, device=device).normal_(0.0, d ** -0.5))
        if weight.shape != (V, d):
            raise ValueError("weight has shape %s, expected [%d, %d]" % (tuple(weight.shape), V, d))
        self.weight = weight

    def forward(self, x, labels):
        return VocabLossFunction.apply(x, self.weight, labels)


def clip_gradients(parameters, max_norm, masters=None, eps=1e-6):
    """Scales the gradients of `parameters` so that their common norm is at most max_norm
    (block.grad_clip) and returns the norm of before, a 0-d tensor.  With `masters`, a
    list of fp32 tensors of the parameters' shapes and in their order, the gradients are left
    alone and the masters' .grad get the scaled ones.  Parameters without a gradient are left out
    (their master's .grad becomes None)."""
    parameters = list(parameters)
    grads = [p.grad for p in parameters if p.grad is not None]
    if masters is None:
        return block.grad_clip(grads, max_norm, eps=eps)
    masters = list(masters)
    if len(masters) != len(parameters):
        raise ValueError("%d masters for %d parameters" % (len(masters), len(parameters)))
    for i, (p, m) in enumerate(zip(parameters, masters)):
        if m.shape != p.shape or m.dtype != torch.float32 or m.device != p.device:
            raise ValueError("master %d is %s %s on %s, expected float32 %s on %s" %
                             (i, m.dtype, tuple(m.shape), m.device, tuple(p.shape), p.device))
    new = [None if p.grad is None else m.grad if m.grad is not None and m.grad.stride() == p.grad.stride() else
           torch.empty_like(p.grad, dtype=torch.float32) for p, m in zip(parameters, masters)]
    norm = block.grad_clip(grads, max_norm, out=[g for g in new if g is not None], eps=eps)
    for m, g in zip(masters, new):      # a refused call has left them as they were
        m.grad = g
    return norm
