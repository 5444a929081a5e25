"""Float64 definitions of the losses on token log probabilities and of orthogonalised updates.  One
sequence, pair, token or matrix after the other, sharing nothing with the kernels."""
from __future__ import annotations

import math

import numpy as np


def spans(shape, offsets=None):
    """(first, end) of each sequence in the flattened tokens."""
    if offsets is None:
        S, L = shape
        return [(s * L, (s + 1) * L) for s in range(S)]
    return [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


def _live(n, where, mask):
    """Whether each token counts: it is some sequence's, and its mask is set."""
    live = np.zeros(n, bool)
    for a, b in where:
        live[a:b] = True
    return live if mask is None else live & np.asarray(mask).reshape(-1)


def _softplus(v):
    if v > 0:
        return v + math.log1p(math.exp(-v))
    return math.log1p(math.exp(v))


def preference_value(kind, h, beta, smoothing=0.0):
    if kind == "sigmoid":
        return (1 - smoothing) * _softplus(-h) + smoothing * _softplus(h)
    if kind == "hinge":
        return max(0.0, 1.0 - h)
    return ((h - 0.5) / beta) ** 2


def preference_slope(kind, h, beta, smoothing=0.0):
    if kind == "sigmoid":
        return smoothing - (1 / (1 + math.exp(h)) if h < 700 else 0.0)
    if kind == "hinge":
        return -1.0 if h < 1 else 0.0
    return 2 * (h - 0.5) / beta ** 2


def preference_loss(logp, chosen, rejected, where, ref=None, mask=None, kind="sigmoid", beta=0.1,
                    margin=0.0, smoothing=0.0, normalize=False):
    """(loss, score, logit, count); logp and ref flat, `where` as spans() gives it."""
    logp = np.asarray(logp, np.float64).reshape(-1)
    live = _live(logp.size, where, mask)
    score, count = np.zeros(len(where)), np.zeros(len(where))
    for s, (a, b) in enumerate(where):
        at = np.arange(a, b)[live[a:b]]
        v = logp[at] if ref is None else logp[at] - np.asarray(ref, np.float64).reshape(-1)[at]
        count[s] = at.size
        score[s] = beta * math.fsum(v) / (max(at.size, 1) if normalize else 1)
    loss, logit = np.zeros(len(chosen)), np.zeros(len(chosen))
    for p, (c, r) in enumerate(zip(chosen, rejected)):
        if 0 <= c < len(where) and 0 <= r < len(where):
            logit[p] = score[c] - score[r] - margin
            loss[p] = preference_value(kind, logit[p], beta, smoothing)
    return loss, score, logit, count


def preference_backward(grad_loss, logit, count, chosen, rejected, where, n, mask=None,
                        kind="sigmoid", beta=0.1, smoothing=0.0, normalize=False):
    """grad_logp, flat."""
    per = np.zeros(len(where))
    for g, h, c, r in zip(grad_loss, logit, chosen, rejected):
        if 0 <= c < len(where) and 0 <= r < len(where):
            v = beta * float(g) * preference_slope(kind, float(h), beta, smoothing)
            per[c] += v
            per[r] -= v
    live, grad = _live(n, where, mask), np.zeros(n)
    for s, (a, b) in enumerate(where):
        grad[a:b] = per[s] / (max(count[s], 1) if normalize else 1)
    return np.where(live, grad, 0.0)


def policy_terms(logp, old, adv, ref=None, clip=(0.2, 0.2), dual=math.inf, kl_coef=0.0):
    """(loss, slope, kl, held, ratio) of one token."""
    ratio = math.exp(logp - old)
    if adv >= 0:
        bounded = min(ratio, 1 + clip[1])
    else:
        bounded = min(max(ratio, 1 - clip[0]), dual)
    held = bounded != ratio and adv != 0
    loss, slope = -adv * bounded, 0.0 if held else -adv * ratio
    kl = 0.0
    if ref is not None:
        d = ref - logp
        kl = math.expm1(d) - d
        loss += kl_coef * kl
        slope -= kl_coef * math.expm1(d)
    return loss, slope, kl, float(held), ratio


def policy_loss(logp, old, adv, where, ref=None, mask=None, clip=(0.2, 0.2), dual=math.inf,
                kl_coef=0.0, reduce="token", denominator=None):
    """(loss, stats, weight, grad for a gradient of 1); adv per token, or one per sequence."""
    flat = [None if t is None else np.asarray(t, np.float64).reshape(-1) for t in (logp, old, adv, ref)]
    logp, old, adv, ref = flat
    n = logp.size
    live = _live(n, where, mask)
    if adv.size != n:
        spread = np.zeros(n)
        for s, (a, b) in enumerate(where):
            spread[a:b] = adv[s]
        adv = spread
    terms = np.zeros((n, 5))
    for t in np.nonzero(live)[0]:
        terms[t] = policy_terms(logp[t], old[t], adv[t], None if ref is None else ref[t], clip, dual,
                                kl_coef)
    total = int(live.sum())
    factor = np.zeros(n)
    if reduce == "token":
        weight = np.array([1.0 / (denominator or max(total, 1))])
        factor[:] = weight[0]
    else:
        counts = [int(live[a:b].sum()) for a, b in where]
        by = denominator or max(1, sum(c > 0 for c in counts))
        weight = np.array([1.0 / (c * by) if c else 0.0 for c in counts])
        for w, (a, b) in zip(weight, where):
            factor[a:b] = w
    stats = np.array([*(terms[live][:, 2:].sum(0) / max(total, 1)), total])
    return math.fsum(factor[live] * terms[live][:, 0]), stats, weight, np.where(live, factor * terms[:, 1], 0.0)


def orthogonalize(x, coefficients, eps=1e-7):
    """The iteration's last X of one matrix."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        x = x / (np.sqrt((x * x).sum()) + eps)
        for a, b, c in coefficients:
            if x.shape[0] <= x.shape[1]:
                s = x @ x.T
                x = a * x + (b * s + c * (s @ s)) @ x
            else:
                s = x.T @ x
                x = a * x + x @ (b * s + c * (s @ s))
    return x


def muon_step(p, g, m, lr, momentum, nesterov, weight_decay, coefficients, eps, factor):
    """(p, m) after a step."""
    p, g, m = (np.asarray(t, np.float64) for t in (p, g, m))
    m = momentum * m + (1 - momentum) * g
    u = momentum * m + (1 - momentum) * g if nesterov else m
    return p * (1 - lr * weight_decay) - lr * factor * orthogonalize(u, coefficients, eps), m
