"""Float64 definitions of the operators around the adapted layers: layer norm, token log
probabilities and AdamW.  Dense, one step after the other, sharing nothing with the kernels."""
from __future__ import annotations

import numpy as np

STATE_BLOCK = 128


def layernorm(x, w, b, eps):
    """(y, mean, rstd) over the rows of x; w and b may be None."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    rstd = 1.0 / np.sqrt(var + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean, rstd


def layernorm_backward(gy, x, w, mean, rstd):
    """(gx, gw, gb) for mean and rstd as the forward returned them."""
    gy, x = np.asarray(gy, np.float64), np.asarray(x, np.float64)
    xhat = (x - mean[:, None]) * rstd[:, None]
    h = gy if w is None else gy * w
    gx = rstd[:, None] * (h - h.mean(axis=1, keepdims=True)
                          - xhat * (h * xhat).mean(axis=1, keepdims=True))
    return gx, (gy * xhat).sum(axis=0), gy.sum(axis=0)


def token_logprob(z, y, scale=1.0, top=0):
    """(logp, entropy, lse, top_logp, top_index); rows whose target is outside the vocabulary
    give zeros (index -1), rows with nothing left logp = lse = -inf and entropy 0."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    logp, entropy, lse = np.zeros(T), np.zeros(T), np.zeros(T)
    top_logp, top_index = np.zeros((T, top)), np.full((T, top), -1, np.int64)
    for t in range(T):
        if not 0 <= y[t] < V:
            continue
        order = np.lexsort((np.arange(V), -z[t]))     # value falling, then index rising
        if np.isnan(z[t]).any():                       # NaN first
            order = np.lexsort((np.arange(V), np.where(np.isnan(z[t]), 0.0, -z[t]),
                                ~np.isnan(z[t])))
        top_index[t] = order[:top]
        m = np.max(z[t])
        if m == -np.inf:
            logp[t] = lse[t] = -np.inf
            top_logp[t] = -np.inf
            continue
        with np.errstate(invalid="ignore"):
            l = (z[t] - m) * scale
            e = np.exp(l)
            s = e.sum()
            lp = l - np.log(s)
            p = e / s
            logp[t] = lp[y[t]]
            entropy[t] = -np.sum(np.where(p > 0, p * lp, 0.0)) if not np.isnan(s) else np.nan
            lse[t] = m * scale + np.log(s)
            top_logp[t] = lp[top_index[t]]
    return logp, entropy, lse, top_logp, top_index


def token_logprob_backward(ga, gh, z, y, scale=1.0):
    """d(sum ga logp + gh entropy)/dz."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    out = np.zeros((T, V))
    for t in range(T):
        m = np.max(z[t])
        if not 0 <= y[t] < V or m == -np.inf:
            continue
        with np.errstate(invalid="ignore"):
            l = (z[t] - m) * scale
            lp = l - np.log(np.exp(l).sum())
            p = np.exp(lp)
            H = -np.sum(np.where(p > 0, p * lp, 0.0))
            g = -ga[t] * p - gh[t] * np.where(p > 0, p * (lp + H), 0.0 * p)
            g[y[t]] += ga[t]
        out[t] = scale * g
    return out


def adamw(p, g, m, v, *, step, lr, beta1, beta2, eps, weight_decay, factor=1.0):
    """(p, m, v) after one step."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    g = g * factor
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mhat, vhat = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    p = p - lr * weight_decay * p - lr * mhat / (np.sqrt(vhat) + eps)
    return p, m, v


def clip_factor(grads, max_norm):
    norm = np.sqrt(sum(float(np.sum(np.asarray(g, np.float64) ** 2)) for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def state_scales(v):
    """Largest magnitude of each block of 128."""
    v = np.abs(np.asarray(v, np.float64).ravel())
    n = -(-v.size // STATE_BLOCK)
    pad = np.zeros(n * STATE_BLOCK)
    pad[:v.size] = v
    return pad.reshape(n, STATE_BLOCK).max(axis=1)


def state_values(codes, scales):
    """First moments of int8 codes; SQUARE ROOTS of second moments of uint8 codes."""
    c = np.asarray(codes, np.float64).ravel()
    a = np.repeat(np.asarray(scales, np.float64), STATE_BLOCK)[:c.size]
    most = 127.0 if codes.dtype == np.int8 else 255.0
    return np.sign(c) * a * (c / most) ** 2


def state_positions(v, scales, most):
    """Where |values| lie on the scale of codes, as real numbers: most * sqrt(|v| / scale)."""
    v = np.abs(np.asarray(v, np.float64).ravel())
    a = np.repeat(np.asarray(scales, np.float64), STATE_BLOCK)[:v.size]
    return most * np.sqrt(np.divide(v, a, out=np.zeros_like(v), where=a > 0))
