"""DoRA and DVoRA linear layers, layer norm, token log probabilities and the losses on them on top of
the C ABI (autograd glue only).

Forward saves norm, xs = s (x A^T) and y for the backward; the norm is
detached there (DoRA reading notes, Sec. 3.4).  DVoRA (Sec. 3.5) runs the same
entry points with B = diag(b) B_shared diag(d).
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import ops


class DoRAFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W0, A, B, m, s, flags):
        y, norm, xs = ops.dora_forward(x, W0, A, B, m, s, flags=flags)
        ctx.s = s
        ctx.flags = flags
        ctx.save_for_backward(x, W0, A, B, m, norm, xs, y)
        ctx.mark_non_differentiable(norm)
        return y, norm

    @staticmethod
    def backward(ctx, gy, _gnorm):
        x, W0, A, B, m, norm, xs, y = ctx.saved_tensors
        need = tuple(n for n, k in (("x", 0), ("A", 2), ("B", 3), ("m", 4))
                     if ctx.needs_input_grad[k])
        gx, gA, gB, gm = ops.dora_backward(gy.contiguous(), x, W0, A, B, m, norm, xs, y, ctx.s,
                                           need=need, flags=ctx.flags)
        if gm is not None:
            gm = gm.to(m.dtype)
        return gx, None, gA, gB, gm, None, None


class DoRALinear(torch.nn.Module):
    """y = (m / ||W0 + s B A||_row) * (x W0^T + s (x A^T) B^T), W0 frozen.

    Initialised as DoRA starts training (DoRA reading notes, Algorithm 1):
    m = row norms of W0, A Kaiming-uniform, B = 0.
    """

    def __init__(self, weight: torch.Tensor, r: int, s: float = 2.0, flags: int = 0):
        super().__init__()
        d_out, d_in = weight.shape
        dev, dt = weight.device, weight.dtype
        self.register_buffer("W0", weight.detach().contiguous())
        self.A = torch.nn.Parameter(torch.empty(r, d_in, device=dev, dtype=dt))
        torch.nn.init.kaiming_uniform_(self.A, a=math.sqrt(5))
        self.B = torch.nn.Parameter(torch.zeros(d_out, r, device=dev, dtype=dt))
        self.m = torch.nn.Parameter(torch.empty(d_out, device=dev, dtype=dt))
        with torch.no_grad():
            self.m.copy_(ops.dora_norm(self.W0, self.A, self.B, s).to(dt))
        self.s = float(s)
        self.flags = int(flags)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        lead = x.shape[:-1]
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        y, _ = DoRAFunction.apply(x2, self.W0, self.A, self.B, self.m, self.s, self.flags)
        return y.reshape(*lead, y.shape[-1])


class DVoRAFunction(torch.autograd.Function):
    """DoRA with VeRA's direction update: A_shared, B_shared frozen; b, d, m trained."""

    @staticmethod
    def forward(ctx, x, W0, A_sh, B_sh, b, d, m, s, flags):
        Be = ops.dora_vera_scale(B_sh, b, d)
        y, norm, xs = ops.dora_forward(x, W0, A_sh, Be, m, s, flags=flags)
        ctx.s = s
        ctx.flags = flags
        ctx.save_for_backward(x, W0, A_sh, B_sh, b, d, Be, m, norm, xs, y)
        return y

    @staticmethod
    def backward(ctx, gy):
        x, W0, A_sh, B_sh, b, d, Be, m, norm, xs, y = ctx.saved_tensors
        want_vec = ctx.needs_input_grad[4] or ctx.needs_input_grad[5]
        need = tuple(n for n, ok in (("x", ctx.needs_input_grad[0]), ("B", want_vec),
                                      ("m", ctx.needs_input_grad[6])) if ok)
        gx, _, gBe, gm = ops.dora_backward(gy.contiguous(), x, W0, A_sh, Be, m, norm, xs, y, ctx.s,
                                           need=need, flags=ctx.flags)
        gb = gd = None
        if want_vec:
            gb, gd = ops.dora_vera_grads(gBe, B_sh, b, d)
        if gm is not None:
            gm = gm.to(m.dtype)
        return gx, None, None, None, gb, gd, gm, None, None


class DVoRALinear(torch.nn.Module):
    """DVoRA layer: y = (m / ||V'||_row) x V'^T, V' = W0 + s diag(b) B_sh diag(d) A_sh.

    A_shared [r, d_in] and B_shared [d_out, r] are frozen (shared by every layer
    of a model); the trainable vectors start at b = 0 (the update starts at zero,
    as DoRA's B = 0 does) and d = d_init, with m = ||W0_i||.
    """

    def __init__(self, weight, A_shared, B_shared, s: float = 1.0, d_init: float = 0.1,
                 flags: int = 0):
        super().__init__()
        d_out, d_in = weight.shape
        r = A_shared.shape[0]
        dev, dt = weight.device, weight.dtype
        self.register_buffer("W0", weight.detach().contiguous())
        self.register_buffer("A_shared", A_shared.detach().contiguous())
        self.register_buffer("B_shared", B_shared.detach().contiguous())
        self.b = torch.nn.Parameter(torch.zeros(d_out, device=dev, dtype=dt))
        self.d = torch.nn.Parameter(torch.full((r,), float(d_init), device=dev, dtype=dt))
        self.m = torch.nn.Parameter(torch.empty(d_out, device=dev, dtype=dt))
        with torch.no_grad():
            Be = ops.dora_vera_scale(self.B_shared, self.b, self.d)
            self.m.copy_(ops.dora_norm(self.W0, self.A_shared, Be, s).to(dt))
        self.s = float(s)
        self.flags = int(flags)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        lead = x.shape[:-1]
        x2 = x.reshape(-1, x.shape[-1]).contiguous()
        y = DVoRAFunction.apply(x2, self.W0, self.A_shared, self.B_shared, self.b, self.d, self.m,
                                self.s, self.flags)
        return y.reshape(*lead, y.shape[-1])


def _as_rows(x):
    """x as [rows, width], copied if rows are not contiguous or overlap (a broadcast input's)."""
    x2 = x.reshape(-1, x.shape[-1])
    if x2.stride(1) != 1 or (x2.shape[0] > 1 and x2.stride(0) < x2.shape[1]):
        x2 = x2.contiguous()
    return x2


class LayerNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = ops.dora_layernorm(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = tuple(n for n, k in (("x", 0), ("weight", 1), ("bias", 2)) if ctx.needs_input_grad[k])
        gx, gw, gb = ops.dora_layernorm_backward(gy.contiguous(), x, weight, mean, rstd, need=need)
        return gx, gw, gb, None


class LayerNorm(torch.nn.Module):
    """y = weight (x - mean) / sqrt(var + eps) + bias over the last dimension of x.

    weight and bias may be frozen (``requires_grad_(False)``): their gradients are then not formed.
    """

    def __init__(self, width: int, eps: float = 1e-5, bias: bool = True, device=None, dtype=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(width, device=device, dtype=dtype)) if bias else None
        self.eps = float(eps)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        x2 = _as_rows(x)
        return LayerNormFunction.apply(x2, self.weight, self.bias, self.eps).reshape(x.shape)


class TokenLogProbFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, scale, top):
        logp, entropy, lse, top_logp, top_index = ops.dora_token_logprob(logits, targets, scale=scale,
                                                                         top=top)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(logits, targets, lse, entropy)
        if top:
            ctx.mark_non_differentiable(top_logp, top_index)
        return logp, entropy, top_logp, top_index

    @staticmethod
    @once_differentiable
    def backward(ctx, g_logp, g_entropy, _g_top, _g_index):
        if g_logp is None and g_entropy is None:
            return None, None, None, None
        logits, targets, lse, entropy = ctx.saved_tensors
        g = [None if t is None else t.contiguous() for t in (g_logp, g_entropy)]
        return ops.dora_token_logprob_backward(g[0], g[1], logits, targets, lse, entropy,
                                               scale=ctx.scale), None, None, None


def token_logprob(logits: torch.Tensor, targets: torch.Tensor, *, scale: float = 1.0, top: int = 0):
    """Log probability of each target under softmax(scale * logits) and the entropy of that
    distribution, differentiable in the logits; with ``top`` > 0 also the likeliest tokens.

    logits [..., vocab], targets int64 [...] of the same leading shape.  Returns (logp, entropy,
    top_logp, top_index), the first two float32 [...], the others [..., top] or None.  Targets
    outside [0, vocab) (-100, say) give zeros and no gradient.
    """
    lead = targets.shape
    if logits.dim() < 1 or logits.shape[:-1] != lead:
        raise ValueError(f"targets have shape {tuple(lead)}, expected {tuple(logits.shape[:-1])}")
    z = _as_rows(logits)
    logp, entropy, top_logp, top_index = TokenLogProbFunction.apply(z, targets.reshape(-1).contiguous(),
                                                                    float(scale), int(top))
    if top:
        top_logp, top_index = top_logp.reshape(*lead, top), top_index.reshape(*lead, top)
    return logp.reshape(lead), entropy.reshape(lead), top_logp, top_index


def _constants(**tensors):
    """Refuses tensors that want a gradient which these losses do not form."""
    for name, t in tensors.items():
        if t is not None and t.requires_grad:
            raise ValueError(f"{name} is a constant of this loss: detach it")


def _contiguous(*tensors):
    return [None if t is None else t.contiguous() for t in tensors]


class PreferenceLossFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, ref_logp, chosen, rejected, mask, offsets, how):
        loss, score, logit, count = ops.dora_preference_loss(logp, chosen, rejected, ref_logp=ref_logp,
                                                             mask=mask, offsets=offsets, **how)
        ctx.shape, ctx.how = logp.shape, how
        ctx.save_for_backward(logit, count, chosen, rejected, mask, offsets)
        ctx.mark_non_differentiable(score)
        return loss, score

    @staticmethod
    @once_differentiable
    def backward(ctx, g_loss, _g_score):
        logit, count, chosen, rejected, mask, offsets = ctx.saved_tensors
        g = ops.dora_preference_loss_backward(g_loss.contiguous(), logit, count, chosen, rejected,
                                              shape=ctx.shape, mask=mask, offsets=offsets, **ctx.how)
        return g, None, None, None, None, None, None


def preference_loss(logp: torch.Tensor, chosen: torch.Tensor, rejected: torch.Tensor, *, ref_logp=None,
                    mask=None, offsets=None, kind: str = "sigmoid", beta: float = 0.1,
                    margin: float = 0.0, smoothing: float = 0.0, normalize: bool = False):
    """Loss of pairs of sequences, the first of which is preferred, differentiable in ``logp``.

    logp, ref_logp: token log probabilities as ``token_logprob`` gives them, float32 [sequences,
    length] or, with ``offsets`` (int64 [sequences + 1]), packed [tokens]; chosen, rejected: int64
    [pairs], the sequences of each pair.  ``mask`` (bool) tells the tokens that count, ``normalize``
    takes means over them instead of sums.  ``kind`` is sigmoid (with ``smoothing``, the share of
    labels taken to be wrong), hinge or square.

    Returns (loss, score): float32 [pairs], and float32 [sequences] without gradient, beta times a
    sequence's log ratio.
    """
    _constants(ref_logp=ref_logp)
    how = dict(kind=kind, beta=beta, margin=margin, smoothing=smoothing, normalize=normalize)
    logp, ref_logp, chosen, rejected, mask, offsets = _contiguous(logp, ref_logp, chosen, rejected,
                                                                  mask, offsets)
    return PreferenceLossFunction.apply(logp, ref_logp, chosen, rejected, mask, offsets, how)


class PolicyLossFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logp, old_logp, advantages, ref_logp, mask, offsets, how):
        loss, stats, weight = ops.dora_policy_loss(logp, old_logp, advantages, ref_logp=ref_logp,
                                                   mask=mask, offsets=offsets, **how)
        ctx.how = how
        ctx.save_for_backward(weight, logp, old_logp, advantages, ref_logp, mask, offsets)
        ctx.mark_non_differentiable(stats)
        return loss, stats

    @staticmethod
    @once_differentiable
    def backward(ctx, g_loss, _g_stats):
        weight, logp, old_logp, advantages, ref_logp, mask, offsets = ctx.saved_tensors
        g = ops.dora_policy_loss_backward(g_loss.contiguous(), weight, logp, old_logp, advantages,
                                          ref_logp=ref_logp, mask=mask, offsets=offsets, **ctx.how)
        return g, None, None, None, None, None, None


def policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantages: torch.Tensor, *, ref_logp=None,
                mask=None, offsets=None, clip=(0.2, 0.2), dual_clip=None, kl_coef: float = 0.0,
                reduce: str = "token", denominator=None, per_sequence=None):
    """Clipped policy loss on token log probabilities, differentiable in ``logp``.

    logp, old_logp, ref_logp: float32 [sequences, length] or, with ``offsets`` (int64 [sequences +
    1]), packed [tokens]; advantages: float32, of logp's shape or [sequences].  ``per_sequence`` (bool)
    says which of both they are, and has to where a packed batch may have as many tokens as sequences:
    without it advantages that fit both are the tokens'.  ``mask`` (bool) tells the tokens that count.
    The ratio exp(logp - old_logp) is bounded by 1 - clip[0] and 1 + clip[1]
    (and by ``dual_clip`` where the advantage is negative); ``kl_coef`` weighs the divergence
    exp(d) - 1 - d, d = ref_logp - logp.  ``reduce`` is token (mean over tokens) or sequence (mean
    over sequences of their means); ``denominator`` replaces the number that is divided by.

    Returns (loss, stats): a scalar, and float32 [4] without gradient: mean divergence, share of
    tokens held by a bound, mean ratio, number of counted tokens.
    """
    _constants(old_logp=old_logp, advantages=advantages, ref_logp=ref_logp)
    how = dict(clip=clip, dual_clip=dual_clip, kl_coef=kl_coef, reduce=reduce, denominator=denominator,
               per_sequence=per_sequence)
    logp, old_logp, advantages, ref_logp, mask, offsets = _contiguous(logp, old_logp, advantages,
                                                                      ref_logp, mask, offsets)
    return PolicyLossFunction.apply(logp, old_logp, advantages, ref_logp, mask, offsets, how)
