"""Thin torch binding of libdora.so: same names as the C ABI.

Only argument marshalling happens here: tensors are checked for device,
dtype, shape and contiguity, output and workspace buffers are allocated by
torch's caching allocator (the library allocates nothing), and the raw device
pointers plus torch's current HIP stream are passed to the library.  Every
step of the computation runs in the library's kernels.
"""
from __future__ import annotations

import bisect
import ctypes
import functools
import json

import torch

from . import _lib
from ._lib import DoraError, FLAG_EXACT_NORM_GRAD, FLAG_SEPARATE_COMPOSE  # noqa: F401

_DT = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev):
    # the handle alone: torch.cuda.current_stream builds a Stream object around it (2 us a call)
    return torch._C._cuda_getCurrentRawStream(dev.index)


_bind = None


def _compiled():
    """The compiled short way of the small calls (csrc/bind.cpp), with the library's addresses.
    Its functions return None where the checked way below has to look closer."""
    global _bind
    if _bind is None:
        try:
            from . import _bind as mod
        except ImportError as e:
            raise ImportError("_bind.so is missing: build it with "
                              "`python -m parameter_efficient_fine_dora_amd.build`") from e
        L = _lib.lib()
        mod.init(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in (
            "dora_layernorm_forward", "dora_layernorm_backward", "dora_layernorm_workspace_bytes",
            "dora_token_logprob_forward", "dora_token_logprob_backward",
            "dora_token_logprob_workspace_bytes", "dora_grad_norm", "dora_adamw_step",
            "dora_adamw_dequantize", "dora_preference_forward", "dora_preference_backward",
            "dora_preference_workspace_bytes", "dora_policy_forward", "dora_policy_backward",
            "dora_policy_workspace_bytes", "dora_orthogonalize",
            "dora_orthogonalize_workspace_bytes", "dora_muon_step")))
        _bind = mod
    return _bind


def _on_gpu(t):
    return isinstance(t, torch.Tensor) and t.is_cuda


def _need(t, name, dtype=None, shape=None, dev=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (HIP) tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _layer_dtype(W0):
    if W0.dtype not in _DT:
        raise ValueError(f"unsupported dtype {W0.dtype}; use float32 or bfloat16")
    return _DT[W0.dtype]


def _ws(sh, op, dev, workspace):
    nbytes = _lib.workspace_bytes(sh, op)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    return workspace, workspace.numel() * workspace.element_size()


def _check(rc, what):
    if rc != 0:
        raise DoraError(rc, what)


def workspace_bytes(d_out, d_in, r, tokens, dtype, op, flags=0) -> int:
    dt = _DT[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return _lib.workspace_bytes(_lib.shape(d_out, d_in, r, tokens, dt, 1.0, flags), op)


def dora_norm(W0, A, B, s, *, out=None, workspace=None, flags=0):
    """Row norms ||W0_i + s (BA)_i|| (float32 [d_out]) by the factored method."""
    dev = W0.device
    dt = W0.dtype
    d_out, d_in = W0.shape
    r = A.shape[0]
    _need(W0, "W0", dt, (d_out, d_in))
    _need(A, "A", dt, (r, d_in), dev)
    _need(B, "B", dt, (d_out, r), dev)
    sh = _lib.shape(d_out, d_in, r, 0, _layer_dtype(W0), s, flags)
    if out is None:
        out = torch.empty(d_out, dtype=torch.float32, device=dev)
    _need(out, "out", torch.float32, (d_out,), dev)
    ws, nb = _ws(sh, _lib.OP_NORM, dev, workspace)
    _check(_lib.lib().dora_norm(ctypes.byref(sh), _ptr(W0), _ptr(A), _ptr(B), _ptr(out), _ptr(ws),
                                nb, _stream(dev)), "dora_norm")
    return out


def dora_forward(x, W0, A, B, m, s, *, y=None, norm_out=None, xs_out=None, keep_xs=True,
                 workspace=None, flags=0):
    """DoRA linear forward.  Returns (y [T, d_out], norm [d_out] f32, xs [T, r] or None)."""
    dev = W0.device
    dt = W0.dtype
    d_out, d_in = W0.shape
    r = A.shape[0]
    T = x.shape[0]
    _need(W0, "W0", dt)
    _need(x, "x", dt, (T, d_in), dev)
    _need(A, "A", dt, (r, d_in), dev)
    _need(B, "B", dt, (d_out, r), dev)
    _need(m, "m", dt, (d_out,), dev)
    sh = _lib.shape(d_out, d_in, r, T, _layer_dtype(W0), s, flags)
    if y is None:
        y = torch.empty(T, d_out, dtype=dt, device=dev)
    if norm_out is None:
        norm_out = torch.empty(d_out, dtype=torch.float32, device=dev)
    if xs_out is None and keep_xs:
        xs_out = torch.empty(T, r, dtype=dt, device=dev)
    _need(y, "y", dt, (T, d_out), dev)
    _need(norm_out, "norm_out", torch.float32, (d_out,), dev)
    if xs_out is not None:
        _need(xs_out, "xs_out", dt, (T, r), dev)
    ws, nb = _ws(sh, _lib.OP_FORWARD, dev, workspace)
    _check(_lib.lib().dora_forward(ctypes.byref(sh), _ptr(x), _ptr(W0), _ptr(A), _ptr(B), _ptr(m),
                                   _ptr(y), _ptr(norm_out), _ptr(xs_out), _ptr(ws), nb,
                                   _stream(dev)), "dora_forward")
    return y, norm_out, xs_out


def dora_forward_noalloc(x, W0, A, B, m, s, *, y=None, norm_out=None, xs_out=None, flags=0):
    """dora_forward on the library's static workspace (no workspace argument; the
    library allocates nothing).  Outputs not given are allocated here by torch,
    before the call.  Returns (y, norm, xs or None)."""
    dev = W0.device
    dt = W0.dtype
    d_out, d_in = W0.shape
    r = A.shape[0]
    T = x.shape[0]
    _need(W0, "W0", dt)
    _need(x, "x", dt, (T, d_in), dev)
    _need(A, "A", dt, (r, d_in), dev)
    _need(B, "B", dt, (d_out, r), dev)
    _need(m, "m", dt, (d_out,), dev)
    sh = _lib.shape(d_out, d_in, r, T, _layer_dtype(W0), s, flags)
    if y is None:
        y = torch.empty(T, d_out, dtype=dt, device=dev)
    if norm_out is None:
        norm_out = torch.empty(d_out, dtype=torch.float32, device=dev)
    _need(y, "y", dt, (T, d_out), dev)
    _need(norm_out, "norm_out", torch.float32, (d_out,), dev)
    if xs_out is not None:
        _need(xs_out, "xs_out", dt, (T, r), dev)
    _check(_lib.lib().dora_forward_noalloc(ctypes.byref(sh), _ptr(x), _ptr(W0), _ptr(A), _ptr(B),
                                           _ptr(m), _ptr(y), _ptr(norm_out), _ptr(xs_out),
                                           _stream(dev)), "dora_forward_noalloc")
    return y, norm_out, xs_out


def dora_backward(grad_y, x, W0, A, B, m, norm, xs, y, s, *, need=("x", "A", "B", "m"),
                  grad_x=None, grad_A=None, grad_B=None, grad_m=None, workspace=None, flags=0):
    """DoRA linear backward with the norm detached.

    Returns (grad_x, grad_A, grad_B, grad_m); entries not in ``need`` are None.
    grad_m is float32.
    """
    dev = W0.device
    dt = W0.dtype
    d_out, d_in = W0.shape
    r = A.shape[0]
    T = x.shape[0]
    _need(grad_y, "grad_y", dt, (T, d_out), dev)
    _need(x, "x", dt, (T, d_in), dev)
    _need(W0, "W0", dt)
    _need(A, "A", dt, (r, d_in), dev)
    _need(B, "B", dt, (d_out, r), dev)
    _need(m, "m", dt, (d_out,), dev)
    _need(norm, "norm", torch.float32, (d_out,), dev)
    _need(y, "y", dt, (T, d_out), dev)
    if xs is not None:
        _need(xs, "xs", dt, (T, r), dev)
    sh = _lib.shape(d_out, d_in, r, T, _layer_dtype(W0), s, flags)
    if "x" in need and grad_x is None:
        grad_x = torch.empty(T, d_in, dtype=dt, device=dev)
    if "A" in need and grad_A is None:
        grad_A = torch.empty(r, d_in, dtype=dt, device=dev)
    if "B" in need and grad_B is None:
        grad_B = torch.empty(d_out, r, dtype=dt, device=dev)
    if "m" in need and grad_m is None:
        grad_m = torch.empty(d_out, dtype=torch.float32, device=dev)
    for t, nm, shp, tdt in ((grad_x, "grad_x", (T, d_in), dt), (grad_A, "grad_A", (r, d_in), dt),
                            (grad_B, "grad_B", (d_out, r), dt),
                            (grad_m, "grad_m", (d_out,), torch.float32)):
        if t is not None:
            _need(t, nm, tdt, shp, dev)
    ws, nb = _ws(sh, _lib.OP_BACKWARD, dev, workspace)
    _check(_lib.lib().dora_backward(ctypes.byref(sh), _ptr(grad_y), _ptr(x), _ptr(W0), _ptr(A),
                                    _ptr(B), _ptr(m), _ptr(norm), _ptr(xs), _ptr(y), _ptr(grad_x),
                                    _ptr(grad_A), _ptr(grad_B), _ptr(grad_m), _ptr(ws), nb,
                                    _stream(dev)), "dora_backward")
    return grad_x, grad_A, grad_B, grad_m


def dora_merge(W0, A, B, m, s, *, norm=None, out=None, workspace=None):
    """Merged weight g_i (W0_i + s (BA)_i) for deployment ([d_out, d_in], layer dtype).

    ``norm`` (float32 [d_out], as from dora_norm / dora_forward) is computed when None.
    """
    dev = W0.device
    dt = W0.dtype
    d_out, d_in = W0.shape
    r = A.shape[0]
    _need(W0, "W0", dt)
    _need(A, "A", dt, (r, d_in), dev)
    _need(B, "B", dt, (d_out, r), dev)
    _need(m, "m", dt, (d_out,), dev)
    if norm is not None:
        _need(norm, "norm", torch.float32, (d_out,), dev)
    sh = _lib.shape(d_out, d_in, r, 0, _layer_dtype(W0), s)
    if out is None:
        out = torch.empty(d_out, d_in, dtype=dt, device=dev)
    _need(out, "out", dt, (d_out, d_in), dev)
    ws, nb = _ws(sh, _lib.OP_MERGE, dev, workspace)
    _check(_lib.lib().dora_merge(ctypes.byref(sh), _ptr(W0), _ptr(A), _ptr(B), _ptr(m),
                                 _ptr(norm), _ptr(out), _ptr(ws), nb, _stream(dev)), "dora_merge")
    return out


def dora_vera_scale(B_shared, b, d, *, out=None):
    """DVoRA's effective B = diag(b) B_shared diag(d) ([d_out, r], layer dtype)."""
    dev = B_shared.device
    dt = B_shared.dtype
    d_out, r = B_shared.shape
    _need(b, "b", dt, (d_out,), dev)
    _need(d, "d", dt, (r,), dev)
    sh = _lib.shape(d_out, 8, r, 0, _layer_dtype(B_shared), 1.0)
    if out is None:
        out = torch.empty(d_out, r, dtype=dt, device=dev)
    _need(out, "out", dt, (d_out, r), dev)
    _check(_lib.lib().dora_vera_scale(ctypes.byref(sh), _ptr(B_shared), _ptr(b), _ptr(d), _ptr(out),
                                      _stream(dev)), "dora_vera_scale")
    return out


def dora_vera_grads(grad_B_eff, B_shared, b, d, *, need=("b", "d"), workspace=None):
    """DVoRA's vector gradients from grad_B_eff: returns (grad_b [d_out], grad_d [r])."""
    dev = B_shared.device
    dt = B_shared.dtype
    d_out, r = B_shared.shape
    _need(grad_B_eff, "grad_B_eff", dt, (d_out, r), dev)
    _need(b, "b", dt, (d_out,), dev)
    _need(d, "d", dt, (r,), dev)
    sh = _lib.shape(d_out, 8, r, 0, _layer_dtype(B_shared), 1.0)
    gb = torch.empty(d_out, dtype=dt, device=dev) if "b" in need else None
    gd = torch.empty(r, dtype=dt, device=dev) if "d" in need else None
    ws, nb = _ws(sh, _lib.OP_VERA_GRADS, dev, workspace)
    _check(_lib.lib().dora_vera_grads(ctypes.byref(sh), _ptr(grad_B_eff), _ptr(B_shared), _ptr(b),
                                      _ptr(d), _ptr(gb), _ptr(gd), _ptr(ws), nb, _stream(dev)),
           "dora_vera_grads")
    return gb, gd


def _out(t, name, dtype, shape, dev):
    """An output the caller gave, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    return _need(t, name, dtype, shape, dev)


def _rows(t, name, dtype=None, shape=None, dev=None):
    """Checks a [rows, width] tensor whose rows are contiguous; returns its row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (HIP) tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, has {t.dim()}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if t.shape[0] <= 1:
        return t.shape[1]
    if t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must have rows that do not overlap")
    return t.stride(0)


def _apart(out, name, rows, of):
    """Refuses a contiguous output that shares memory with an input of rows."""
    if not out.numel():
        return
    size, (R, D) = rows.element_size(), rows.shape
    lo = out.data_ptr() - rows.data_ptr()
    hi = lo + out.numel() * out.element_size()
    step = rows.stride(0) * size if R > 1 else D * size
    first = max(0, (lo - D * size) // step + 1)     # the first row that ends past the output's start
    if first < R and first * step < hi:
        raise ValueError(f"{name} must not overlap {of}")


def _given_ws(workspace, dev):
    """Bytes of a workspace that the caller gave: contiguous, on the tensors' device."""
    _need(workspace, "workspace", None, None, dev)
    return workspace.numel() * workspace.element_size()


def dora_layernorm(x, weight=None, bias=None, *, eps=1e-5, y=None, mean=None, rstd=None):
    """Layer norm over the rows of x [rows, width] (rows contiguous, any row stride).

    Returns (y, mean, rstd); mean and rstd are float32 [rows], for the backward.
    """
    if y is None and mean is None and rstd is None and _on_gpu(x):
        out = _compiled().layernorm(x, weight, bias, float(eps), _stream(x.device))
        if out is not None:
            return out
    ld = _rows(x, "x")
    dev, dt = x.device, x.dtype
    R, D = x.shape
    code = _layer_dtype(x)
    for t, nm in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _need(t, nm, dt, (D,), dev)
    y = _out(y, "y", dt, (R, D), dev)
    mean = _out(mean, "mean", torch.float32, (R,), dev)
    rstd = _out(rstd, "rstd", torch.float32, (R,), dev)
    sh = _lib.DoraLayernormShape(R, D, ld, ld, code, eps, 0, 0)
    _check(_lib.lib().dora_layernorm_forward(ctypes.byref(sh), _ptr(x), _ptr(weight), _ptr(bias),
                                             _ptr(y), _ptr(mean), _ptr(rstd), _stream(dev)),
           "dora_layernorm_forward")
    return y, mean, rstd


def dora_layernorm_backward(grad_y, x, weight, mean, rstd, *, need=("x", "weight", "bias"),
                            grad_x=None, grad_weight=None, grad_bias=None, workspace=None):
    """Layer norm backward.  Returns (grad_x, grad_weight, grad_bias), layer dtype; entries not
    in ``need`` are None."""
    if (grad_x is None and grad_weight is None and grad_bias is None and workspace is None
            and _on_gpu(x)):
        out = _compiled().layernorm_backward(grad_y, x, weight, mean, rstd, "x" in need,
                                             "weight" in need, "bias" in need, _stream(x.device))
        if out is not None:
            return out
    ld = _rows(x, "x")
    dev, dt = x.device, x.dtype
    R, D = x.shape
    code = _layer_dtype(x)
    ldg = _rows(grad_y, "grad_y", dt, (R, D), dev)
    if weight is not None:
        _need(weight, "weight", dt, (D,), dev)
    _need(mean, "mean", torch.float32, (R,), dev)
    _need(rstd, "rstd", torch.float32, (R,), dev)
    if grad_x is not None or "x" in need:
        grad_x = _out(grad_x, "grad_x", dt, (R, D), dev)
    if grad_weight is not None or "weight" in need:
        grad_weight = _out(grad_weight, "grad_weight", dt, (D,), dev)
    if grad_bias is not None or "bias" in need:
        grad_bias = _out(grad_bias, "grad_bias", dt, (D,), dev)
    sh = _lib.DoraLayernormShape(R, D, ld, ldg, code, 0.0, 0, 0)
    nb = 0
    if grad_weight is not None or grad_bias is not None or D > _lib.LAYERNORM_NO_WS_WIDTH[code]:
        nb = _lib.lib().dora_layernorm_workspace_bytes(ctypes.byref(sh))
        if workspace is None:
            workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
        nb = _given_ws(workspace, dev)
    _check(_lib.lib().dora_layernorm_backward(ctypes.byref(sh), _ptr(grad_y), _ptr(x), _ptr(weight),
                                              _ptr(mean), _ptr(rstd), _ptr(grad_x),
                                              _ptr(grad_weight), _ptr(grad_bias), _ptr(workspace),
                                              nb, _stream(dev)), "dora_layernorm_backward")
    return grad_x, grad_weight, grad_bias


def dora_token_logprob(logits, targets, *, scale=1.0, top=0, workspace=None):
    """Log probabilities of ``targets`` (int64 [rows]) under softmax(scale * logits) per row.

    Returns (logp, entropy, lse, top_logp, top_index): float32 [rows] each, and, for top > 0, the
    ``top`` likeliest tokens of each row, float32 and int64 [rows, top] (None for top = 0).  Rows
    whose target lies outside [0, vocab) are skipped: zeros, and top_index -1.
    """
    if workspace is None and _on_gpu(logits):
        out = _compiled().token_logprob(logits, targets, float(scale), int(top),
                                        _stream(logits.device))
        if out is not None:
            return out
    ld = _rows(logits, "logits")
    dev = logits.device
    T, V = logits.shape
    _need(targets, "targets", torch.int64, (T,), dev)
    top = int(top) if 0 <= top <= _lib.LOGPROB_MAX_TOP else -1   # ctypes would cut a larger number
    sh = _lib.DoraLogprobShape(T, V, ld, _layer_dtype(logits), top, float(scale), 0)
    logp, entropy, lse = torch.empty(3, T, dtype=torch.float32, device=dev).unbind(0)
    top_logp = top_index = None
    if top > 0:
        top_logp = torch.empty(T, top, dtype=torch.float32, device=dev)
        top_index = torch.empty(T, top, dtype=torch.int64, device=dev)
    nb = _lib.lib().dora_token_logprob_workspace_bytes(ctypes.byref(sh))
    if nb and workspace is None:
        workspace = torch.empty(nb, dtype=torch.uint8, device=dev)
    if workspace is not None:
        nb = _given_ws(workspace, dev)
    _check(_lib.lib().dora_token_logprob_forward(ctypes.byref(sh), _ptr(logits), _ptr(targets),
                                                 _ptr(logp), _ptr(entropy), _ptr(lse),
                                                 _ptr(top_logp), _ptr(top_index), _ptr(workspace),
                                                 nb, _stream(dev)), "dora_token_logprob_forward")
    return logp, entropy, lse, top_logp, top_index


def dora_token_logprob_backward(grad_logp, grad_entropy, logits, targets, lse, entropy, *, scale=1.0,
                                grad_logits=None):
    """Gradient of dora_token_logprob's logp and entropy (either gradient may be None) with respect
    to the logits, [rows, vocab] in their dtype; lse and entropy as it returned them."""
    if grad_logits is None and _on_gpu(logits):
        out = _compiled().token_logprob_backward(grad_logp, grad_entropy, logits, targets, lse,
                                                 entropy, float(scale), _stream(logits.device))
        if out is not None:
            return out
    ld = _rows(logits, "logits")
    dev = logits.device
    T, V = logits.shape
    _need(targets, "targets", torch.int64, (T,), dev)
    for t, nm in ((grad_logp, "grad_logp"), (grad_entropy, "grad_entropy"), (entropy, "entropy")):
        if t is not None:
            _need(t, nm, torch.float32, (T,), dev)
    _need(lse, "lse", torch.float32, (T,), dev)
    grad_logits = _out(grad_logits, "grad_logits", logits.dtype, (T, V), dev)
    _apart(grad_logits, "grad_logits", logits, "logits")
    sh = _lib.DoraLogprobShape(T, V, ld, _layer_dtype(logits), 0, float(scale), 0)
    _check(_lib.lib().dora_token_logprob_backward(ctypes.byref(sh), _ptr(grad_logp),
                                                  _ptr(grad_entropy), _ptr(logits), _ptr(targets),
                                                  _ptr(lse), _ptr(entropy), _ptr(grad_logits),
                                                  _stream(dev)), "dora_token_logprob_backward")
    return grad_logits


def _token_batch(shape, dev, mask, offsets):
    """The sequences of tensors [sequences, length], or of one [tokens] with offsets."""
    if offsets is None:
        if len(shape) != 2:
            raise ValueError(f"log probabilities have shape {tuple(shape)}: two dimensions, or one "
                             "with offsets, are expected")
        S, length = shape
        tokens = S * length
    else:
        if len(shape) != 1:
            raise ValueError(f"log probabilities have shape {tuple(shape)}: one dimension is "
                             "expected with offsets")
        _need(offsets, "offsets", torch.int64, None, dev)
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError(f"offsets have shape {tuple(offsets.shape)}, expected (sequences + 1,)")
        tokens, S, length = shape[0], offsets.numel() - 1, 0
    if mask is not None:
        _need(mask, "mask", torch.bool, shape, dev)
    return _lib.DoraTokenBatch(tokens, S, length, _ptr(offsets), _ptr(mask))


def _choice(value, name, of):
    if value not in of:
        raise ValueError(f"{name} is {value!r}, expected one of {', '.join(of)}")
    return of[value]


def _preference_options(kind, beta, margin, smoothing, normalize):
    return _lib.DoraPreferenceOptions(_choice(kind, "kind", _lib.PREFERENCE_KIND), int(bool(normalize)),
                                      float(beta), float(margin), float(smoothing))


def _some_ws(nbytes, dev, workspace):
    """A workspace of at least `nbytes`, the caller's if there is one; its address and size."""
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    return workspace, _given_ws(workspace, dev)


def dora_preference_loss(logp, chosen, rejected, *, ref_logp=None, mask=None, offsets=None,
                         kind="sigmoid", beta=0.1, margin=0.0, smoothing=0.0, normalize=False,
                         workspace=None):
    """Losses of pairs of sequences by their summed log probabilities, relative to a reference's.

    logp, ref_logp   float32 [sequences, length], or [tokens] with ``offsets`` (int64
                     [sequences + 1]: sequence s has tokens offsets[s] to offsets[s + 1])
    chosen, rejected int64 [pairs]: the sequences of each pair, the preferred one first
    mask             bool, of logp's shape: the tokens that count
    kind             sigmoid, hinge or square; ``smoothing`` is the sigmoid's share of wrong labels
    normalize        means over a sequence's counted tokens instead of sums

    Returns (loss, score, logit, count): float32 [pairs], [sequences], [pairs], [sequences]; score
    is beta times a sequence's sum, logit the difference of two scores less ``margin``.
    """
    if workspace is None and kind in _lib.PREFERENCE_KIND and _on_gpu(logp):
        out = _compiled().preference_loss(logp, ref_logp, chosen, rejected, mask, offsets, float(beta),
                                          float(margin), float(smoothing), _lib.PREFERENCE_KIND[kind],
                                          bool(normalize), _stream(logp.device))
        if out is not None:
            return out
    _need(logp, "logp", torch.float32)
    dev, shape = logp.device, logp.shape
    batch = _token_batch(shape, dev, mask, offsets)
    if ref_logp is not None:
        _need(ref_logp, "ref_logp", torch.float32, shape, dev)
    P, S = _pairs(chosen, rejected, dev), batch.sequences
    how = _preference_options(kind, beta, margin, smoothing, normalize)
    loss, logit = torch.empty(2, P, dtype=torch.float32, device=dev).unbind(0)
    score, count = torch.empty(2, S, dtype=torch.float32, device=dev).unbind(0)
    L = _lib.lib()
    ws, nb = _some_ws(L.dora_preference_workspace_bytes(ctypes.byref(batch)), dev, workspace)
    with torch.cuda.device(dev):   # (the null stream is the current device's)
        _check(L.dora_preference_forward(ctypes.byref(batch), ctypes.byref(how), P, _ptr(logp),
                                         _ptr(ref_logp), _ptr(chosen), _ptr(rejected), _ptr(loss),
                                         _ptr(score), _ptr(logit), _ptr(count), _ptr(ws), nb,
                                         _stream(dev)), "dora_preference_forward")
    return loss, score, logit, count


def _pairs(chosen, rejected, dev):
    _need(chosen, "chosen", torch.int64, None, dev)
    if chosen.dim() != 1:
        raise ValueError(f"chosen must have one dimension, has {chosen.dim()}")
    _need(rejected, "rejected", torch.int64, chosen.shape, dev)
    return chosen.numel()


def dora_preference_loss_backward(grad_loss, logit, count, chosen, rejected, *, shape, mask=None,
                                  offsets=None, kind="sigmoid", beta=0.1, margin=0.0, smoothing=0.0,
                                  normalize=False, grad_logp=None, workspace=None):
    """Gradient of dora_preference_loss's losses with respect to logp (of ``shape``), float32;
    logit and count as it returned them."""
    shape = tuple(shape)
    if grad_logp is None and workspace is None and kind in _lib.PREFERENCE_KIND and _on_gpu(logit):
        out = _compiled().preference_loss_backward(
            grad_loss, logit, count, chosen, rejected, mask, offsets, float(beta), float(margin),
            float(smoothing), _lib.PREFERENCE_KIND[kind], bool(normalize), shape, _stream(logit.device))
        if out is not None:
            return out
    _need(logit, "logit", torch.float32)
    dev = logit.device
    batch = _token_batch(shape, dev, mask, offsets)
    P = _pairs(chosen, rejected, dev)
    _need(logit, "logit", torch.float32, (P,), dev)
    _need(grad_loss, "grad_loss", torch.float32, (P,), dev)
    _need(count, "count", torch.float32, (batch.sequences,), dev)
    how = _preference_options(kind, beta, margin, smoothing, normalize)
    grad_logp = _out(grad_logp, "grad_logp", torch.float32, shape, dev)
    L = _lib.lib()
    ws, nb = _some_ws(L.dora_preference_workspace_bytes(ctypes.byref(batch)), dev, workspace)
    with torch.cuda.device(dev):   # (the null stream is the current device's)
        _check(L.dora_preference_backward(ctypes.byref(batch), ctypes.byref(how), P, _ptr(grad_loss),
                                          _ptr(logit), _ptr(count), _ptr(chosen), _ptr(rejected),
                                          _ptr(grad_logp), _ptr(ws), nb, _stream(dev)),
               "dora_preference_backward")
    return grad_logp


def _policy_numbers(clip, dual_clip, kl_coef, reduce, denominator, ref_logp):
    """The options as the compiled way takes them, or None where they have to be looked at."""
    if reduce not in _lib.POLICY_REDUCE or (kl_coef and ref_logp is None) or denominator == 0:
        return None
    return (float(clip[0]), float(clip[1]), float("inf") if dual_clip is None else float(dual_clip),
            float(kl_coef), 0.0 if denominator is None else float(denominator), _lib.POLICY_REDUCE[reduce])


def _policy_arguments(logp, old_logp, advantages, ref_logp, mask, offsets, clip, dual_clip, kl_coef,
                      reduce, denominator, per_sequence):
    """Checks what both directions of the policy loss take; returns the batch and the options."""
    _need(logp, "logp", torch.float32)
    dev, shape = logp.device, logp.shape
    batch = _token_batch(shape, dev, mask, offsets)
    _need(old_logp, "old_logp", torch.float32, shape, dev)
    if ref_logp is not None:
        _need(ref_logp, "ref_logp", torch.float32, shape, dev)
    elif kl_coef:
        raise ValueError("kl_coef needs ref_logp")
    # unless the caller says: one advantage a token where the shapes agree, else one a sequence
    each = (isinstance(advantages, torch.Tensor) and advantages.shape == shape if per_sequence is None
            else not per_sequence)
    _need(advantages, "advantages", torch.float32, shape if each else (batch.sequences,), dev)
    if denominator is not None and not denominator > 0:
        raise ValueError(f"denominator is {denominator}, expected more than 0")
    return batch, _lib.DoraPolicyOptions(
        float(clip[0]), float(clip[1]), float("inf") if dual_clip is None else float(dual_clip),
        float(kl_coef), 0.0 if denominator is None else float(denominator),
        _choice(reduce, "reduce", _lib.POLICY_REDUCE), int(not each))


def dora_policy_loss(logp, old_logp, advantages, *, ref_logp=None, mask=None, offsets=None,
                     clip=(0.2, 0.2), dual_clip=None, kl_coef=0.0, reduce="token", denominator=None,
                     per_sequence=None, workspace=None):
    """Clipped policy loss of tokens, with ``kl_coef`` times their divergence from a reference.

    logp, old_logp, ref_logp   float32 [sequences, length], or [tokens] with ``offsets`` (int64
                     [sequences + 1])
    advantages       float32, one a token (logp's shape) or one a sequence ([sequences]), as
                     ``per_sequence`` says; by their shape where it is None, and one a token where a
                     packed batch has as many tokens as sequences and the shape does not tell
    mask             bool, of logp's shape: the tokens that count
    clip             the ratio's bounds are 1 - clip[0] and 1 + clip[1]; ``dual_clip`` bounds it from
                     above where the advantage is negative
    reduce           token: sum over tokens / their number; sequence: mean over the sequences of
                     their means.  ``denominator`` takes the place of the number.

    Returns (loss, stats, weight): a float32 scalar; float32 [4], the counted tokens' mean
    divergence, the share of them held by a bound, their mean ratio and their number; the factor of
    each sequence's tokens in the loss, float32 [sequences] or [1], for the backward.
    """
    if workspace is None and _on_gpu(logp):
        fast = _policy_numbers(clip, dual_clip, kl_coef, reduce, denominator, ref_logp)
        out = fast and _compiled().policy_loss(logp, old_logp, advantages, ref_logp, mask, offsets, *fast,
                                               per_sequence, _stream(logp.device))
        if out is not None:
            return out
    batch, how = _policy_arguments(logp, old_logp, advantages, ref_logp, mask, offsets, clip,
                                   dual_clip, kl_coef, reduce, denominator, per_sequence)
    dev = logp.device
    loss = torch.empty((), dtype=torch.float32, device=dev)
    stats = torch.empty(4, dtype=torch.float32, device=dev)
    weight = torch.empty(batch.sequences if how.reduce else 1, dtype=torch.float32, device=dev)
    L = _lib.lib()
    nb = L.dora_policy_workspace_bytes(ctypes.byref(batch), ctypes.byref(how))
    ws, nb = _some_ws(nb, dev, workspace)
    with torch.cuda.device(dev):   # (the null stream is the current device's)
        _check(L.dora_policy_forward(ctypes.byref(batch), ctypes.byref(how), _ptr(logp), _ptr(old_logp),
                                     _ptr(ref_logp), _ptr(advantages), _ptr(loss), _ptr(stats),
                                     _ptr(weight), _ptr(ws), nb, _stream(dev)), "dora_policy_forward")
    return loss, stats, weight


def dora_policy_loss_backward(grad_loss, weight, logp, old_logp, advantages, *, ref_logp=None,
                              mask=None, offsets=None, clip=(0.2, 0.2), dual_clip=None, kl_coef=0.0,
                              reduce="token", denominator=None, per_sequence=None, grad_logp=None):
    """Gradient of dora_policy_loss's loss with respect to logp, float32 of its shape; grad_loss is a
    float32 scalar on the device, weight as the forward returned it, the rest as the forward took it."""
    if grad_logp is None and _on_gpu(logp):
        fast = _policy_numbers(clip, dual_clip, kl_coef, reduce, denominator, ref_logp)
        out = fast and _compiled().policy_loss_backward(logp, old_logp, advantages, ref_logp, mask, offsets,
                                                        *fast, per_sequence, grad_loss, weight,
                                                        _stream(logp.device))
        if out is not None:
            return out
    batch, how = _policy_arguments(logp, old_logp, advantages, ref_logp, mask, offsets, clip,
                                   dual_clip, kl_coef, reduce, denominator, per_sequence)
    dev = logp.device
    if _need(grad_loss, "grad_loss", torch.float32, None, dev).numel() != 1:
        raise ValueError("grad_loss must be one number")
    _need(weight, "weight", torch.float32, (batch.sequences if how.reduce else 1,), dev)
    grad_logp = _out(grad_logp, "grad_logp", torch.float32, logp.shape, dev)
    with torch.cuda.device(dev):   # (the null stream is the current device's)
        _check(_lib.lib().dora_policy_backward(ctypes.byref(batch), ctypes.byref(how), _ptr(grad_loss),
                                               _ptr(weight), _ptr(logp), _ptr(old_logp), _ptr(ref_logp),
                                               _ptr(advantages), _ptr(grad_logp), _stream(dev)),
               "dora_policy_backward")
    return grad_logp


class AdamWPlan:
    """The tensors of an AdamW step, checked once and kept for the steps that follow.

    params         contiguous tensors of one dtype (bf16 or float32) on one device
    exp_avg, exp_avg_sq   the moments, one tensor per parameter: float32 of its size, or 8-bit codes
                   (int8 and uint8) with ``exp_avg_scales`` / ``exp_avg_sq_scales``, float32
                   [ceil(n / 128)] each
    masters        float32 copies of bf16 parameters, or None

    The plan refers to the tensors (they stay alive with it) and writes through them.  A tensor
    whose storage was exchanged since (``p.data = ...``, ``exp_avg.data = ...``) is an error at the
    next step: the table has the old address.
    """

    _STATE_FIELDS = ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "master")

    def __init__(self, params, exp_avg, exp_avg_sq, *, masters=None, exp_avg_scales=None,
                 exp_avg_sq_scales=None):
        params, exp_avg, exp_avg_sq = list(params), list(exp_avg), list(exp_avg_sq)
        if not params:
            raise ValueError("params is empty")
        n = len(params)
        small = exp_avg_scales is not None or exp_avg_sq_scales is not None
        sc1 = None if exp_avg_scales is None else list(exp_avg_scales)
        sc2 = None if exp_avg_sq_scales is None else list(exp_avg_sq_scales)
        mst = None if masters is None else list(masters)
        self.table = (_lib.DoraAdamwTensor * n)()
        self._address = ctypes.addressof(self.table)
        self._lists = (params, exp_avg, exp_avg_sq, sc1, sc2, mst)
        code = _compiled().make_table(*self._lists, self._address)
        if code is None:
            code = self._checked_table(self.table, *self._lists)
        self.param_code = code
        self.params, self.device, self.dtype = params, params[0].device, params[0].dtype
        self.state_bits = 8 if small else 32
        self.norm_bytes = None   # workspace of the gradients' norm, asked for once

    @staticmethod
    def _checked_table(table, params, exp_avg, exp_avg_sq, sc1, sc2, mst):
        """Fills a table tensor by tensor and says what is wrong."""
        n, small = len(params), sc1 is not None
        if small != (sc2 is not None):
            raise ValueError("8-bit states need exp_avg_scales and exp_avg_sq_scales")
        lists = [("exp_avg", exp_avg, torch.int8 if small else torch.float32, False),
                 ("exp_avg_sq", exp_avg_sq, torch.uint8 if small else torch.float32, False),
                 ("exp_avg_scale", sc1, torch.float32, True),
                 ("exp_avg_sq_scale", sc2, torch.float32, True),
                 ("master", mst, torch.float32, False)]
        for nm, lst, _, _ in lists:
            if lst is not None and len(lst) != n:
                raise ValueError(f"{nm} has {len(lst)} tensors, expected {n}")
        _need(params[0], "params[0]")
        dev, dt = params[0].device, params[0].dtype
        code = _layer_dtype(params[0])
        if mst is not None and dt != torch.bfloat16:
            raise ValueError("masters go with bfloat16 params")
        for i, (e, p) in enumerate(zip(table, params)):
            k = _need(p, f"params[{i}]", dt, None, dev).numel()
            e.param, e.n = p.data_ptr(), k
            for nm, lst, tdt, per_block in lists:
                if lst is None:
                    continue
                t = _need(lst[i], f"{nm}[{i}]", tdt, None, dev)
                size = -(-k // _lib.STATE_BLOCK) if per_block else k
                if t.numel() != size:
                    raise ValueError(f"{nm}[{i}] has {t.numel()} elements, expected {size}")
                setattr(e, nm, t.data_ptr())
        written = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), f"{nm}[{i}]")
                         for nm, lst in [("params", params)] + [x[:2] for x in lists] if lst is not None
                         for i, t in enumerate(lst) if t.numel())
        for a, b in zip(written, written[1:]):
            if b[0] < a[1]:
                raise ValueError(f"{a[2]} and {b[2]} share memory: a step writes both")
        return code

    def unchanged(self):
        """Whether every tensor still has the storage it had when the plan was made."""
        return (self.params[0].dtype == self.dtype
                and _compiled().same_table(*self._lists, self._address))

    def _check_storage(self):
        """Says which tensor has another storage than the table's, or another type or size."""
        if [p.data_ptr() for p in self.params] != [e.param or 0 for e in self.table]:
            raise ValueError("a parameter's storage has changed since the plan was made")
        for nm, lst in zip(self._STATE_FIELDS, self._lists[1:]):
            for i, (t, e) in enumerate(zip(lst or (), self.table)):
                if t.data_ptr() != (getattr(e, nm) or 0):
                    raise ValueError(f"{nm}[{i}]'s storage has changed since the plan was made")
        now = (_lib.DoraAdamwTensor * len(self.params))()
        code = self._checked_table(now, *self._lists)
        if code != self.param_code or [e.n for e in now] != [e.n for e in self.table]:
            raise ValueError("a parameter's type or size has changed since the plan was made")

    def _take_grads(self, grads):
        """Checks the gradients and notes where they are; returns their dtype's code."""
        grads = grads if isinstance(grads, list) else list(grads)
        code = _compiled().take_grads(*self._lists, self._address, grads, self.device.index)
        if code is not None and self.params[0].dtype == self.dtype:
            return code
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} params")
        self._check_storage()
        gdt = grads[0].dtype if isinstance(grads[0], torch.Tensor) else None
        if gdt is not None and gdt not in _DT:
            raise ValueError(f"unsupported dtype {gdt}; use float32 or bfloat16")
        for i, (g, e) in enumerate(zip(grads, self.table)):
            _need(g, f"grads[{i}]", gdt, None, self.device)
            if g.numel() != e.n:
                raise ValueError(f"grads[{i}] has {g.numel()} elements, expected {e.n}")
            e.grad = g.data_ptr()
        return _DT[gdt]


def dora_grad_norm(plan, grads, max_norm=1.0, *, workspace=None):
    """Global norm of the gradients of a plan's params and the factor min(1, max_norm / (norm +
    1e-6)) that clips them to ``max_norm``: two float32 scalars on the device."""
    return _grad_norm(plan, plan._take_grads(grads), max_norm, workspace)


def _grad_norm(plan, code, max_norm, workspace):
    L, n = _lib.lib(), len(plan.params)
    if workspace is None:
        if plan.norm_bytes is None:
            plan.norm_bytes = L.dora_grad_norm_workspace_bytes(plan.table, n)
        out = _compiled().grad_norm(plan._address, n, code, float(max_norm), plan.norm_bytes,
                                    plan.params[0], _stream(plan.device))
        if out is not None:
            return out
        workspace = torch.empty(max(plan.norm_bytes, 1), dtype=torch.uint8, device=plan.device)
    norm = torch.empty((), dtype=torch.float32, device=plan.device)
    factor = torch.empty((), dtype=torch.float32, device=plan.device)
    _check(L.dora_grad_norm(plan.table, n, code, float(max_norm), _ptr(norm), _ptr(factor),
                            _ptr(workspace), _given_ws(workspace, plan.device),
                            _stream(plan.device)), "dora_grad_norm")
    return norm, factor


def dora_adamw(plan, grads, *, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
               max_norm=None, grad_scale=None, workspace=None):
    """One AdamW step (``step`` counts from 1) on the tensors of a plan, in place.

    ``grads``: one contiguous tensor per parameter, all bf16 or all float32.  With ``max_norm`` the
    gradients are first clipped by their global norm, which is returned (a float32 scalar on the
    device); ``grad_scale`` is a float32 scalar on the device to multiply them by instead.
    """
    if max_norm is not None and grad_scale is not None:
        raise ValueError("max_norm and grad_scale exclude each other")
    code = plan._take_grads(grads)
    norm = None
    if max_norm is not None:
        norm, grad_scale = _grad_norm(plan, code, max_norm, workspace)
    elif grad_scale is not None:
        if _need(grad_scale, "grad_scale", torch.float32, None, plan.device).numel() != 1:
            raise ValueError("grad_scale must be one number")
    _check(_compiled().adamw_step(plan._address, plan.params, plan.param_code, code,
                                  plan.state_bits, int(step), float(lr), float(betas[0]),
                                  float(betas[1]), float(eps), float(weight_decay), grad_scale,
                                  _stream(plan.device)), "dora_adamw_step")
    return norm


# Newton-Schulz coefficients that take singular values from 2e-3 to 1 to within [0.68, 1.13]
NEWTON_SCHULZ = ((3.4445, -4.7750, 2.0315),) * 5


@functools.lru_cache(maxsize=16)
def _coefficients(coefficients):
    """(array, its address, steps) of ((a, b, c), ...)."""
    flat = [float(v) for abc in coefficients for v in abc]
    if any(len(abc) != 3 for abc in coefficients):
        raise ValueError("coefficients are (a, b, c) for each step")
    array = (ctypes.c_double * max(len(flat), 1))(*flat)
    return array, ctypes.addressof(array), len(flat) // 3


def _iteration(coefficients, eps):
    """The iteration's struct, and the array of coefficients that it points to."""
    array, address, steps = _coefficients(tuple(tuple(abc) for abc in coefficients))
    return _lib.DoraNewtonSchulz(address, steps, 0, float(eps)), array


def dora_orthogonalize(x, *, coefficients=NEWTON_SCHULZ, eps=1e-7, out=None, workspace=None):
    """The orthogonalised matrix (or matrices) of ``x`` by Newton-Schulz products: x / (|x| + eps),
    then a x + (b s + c s^2) x with s = x x^T for each (a, b, c) of ``coefficients``.

    x: a contiguous [rows, cols] tensor, a stack [count, rows, cols], or a list of matrices of any
    sizes, bf16 or float32.  Returns the same kind; ``out`` may be x itself.
    """
    if out is None and workspace is None and _on_gpu(x):
        _held, address, steps = _coefficients(tuple(tuple(abc) for abc in coefficients))
        out = _compiled().orthogonalize(x, address, steps, float(eps), _stream(x.device))
        if out is not None:
            return out
    many = isinstance(x, (list, tuple))
    xs = list(x) if many else [x]
    outs = [None] * len(xs) if out is None else list(out) if many else [out]
    if len(outs) != len(xs):
        raise ValueError(f"out has {len(outs)} tensors, expected {len(xs)}")
    if not xs:
        return []
    _need(xs[0], "x[0]" if many else "x")
    dev, dt = xs[0].device, xs[0].dtype
    code = _layer_dtype(xs[0])
    counts = []
    for i, t in enumerate(xs):
        name = f"x[{i}]" if many else "x"
        _need(t, name, dt, None, dev)
        if t.dim() not in ((2,) if many else (2, 3)):
            raise ValueError(f"{name} has {t.dim()} dimensions, expected a matrix"
                             + ("" if many else " or a stack of them"))
        outs[i] = _out(outs[i], "out", dt, t.shape, dev)
        counts.append(t.shape[0] if t.dim() == 3 else 1)
    if out is not None:
        _disjoint(outs, xs)
    table = (_lib.DoraMatrix * max(sum(counts), 1))()
    size, at = xs[0].element_size(), 0
    for t, o, k in zip(xs, outs, counts):
        rows, cols = t.shape[-2:]
        a, b = t.data_ptr(), o.data_ptr()
        for j in range(k):
            e = table[at]
            e.x, e.out, e.rows, e.cols = a + j * rows * cols * size, b + j * rows * cols * size, rows, cols
            at += 1
    iteration, _held = _iteration(coefficients, eps)
    how = _lib.DoraOrthogonalizeOptions(iteration, code, 0)
    L = _lib.lib()
    nb = L.dora_orthogonalize_workspace_bytes(table, at, ctypes.byref(how))
    ws, nb = _some_ws(nb, dev, workspace)
    with torch.cuda.device(dev):   # (the null stream is the current device's)
        _check(L.dora_orthogonalize(table, at, ctypes.byref(how), _ptr(ws), nb, _stream(dev)),
               "dora_orthogonalize")
    return outs if many else outs[0]


def _disjoint(outs, xs):
    """Refuses outputs that share memory with each other or with an input that is not their own:
    matrices are worked on in any order."""
    spans = []   # (first byte, end, whether it is written)
    for o, x in zip(outs, xs):
        if o.numel():
            size, a, b = o.numel() * o.element_size(), o.data_ptr(), x.data_ptr()
            spans.append((a, a + size, True))
            if a != b:
                spans.append((b, b + size, False))
    end = written = 0
    for lo, hi, write in sorted(spans):
        if lo < (end if write else written):
            raise ValueError("out must not overlap: a matrix may take its own x's place, and no other")
        end, written = max(end, hi), max(written, hi if write else 0)


class MuonPlan:
    """The matrices of a step with orthogonalised updates, checked once and kept for the steps that
    follow.

    params     contiguous matrices of one dtype (bf16 or float32) on one device
    momenta    float32 tensors of their shapes
    masters    float32 copies of bf16 parameters, or None

    The plan refers to the tensors and writes through them.  A tensor whose storage was exchanged
    since is an error at the next step.
    """

    def __init__(self, params, momenta, *, masters=None):
        self.params, self.momenta = list(params), list(momenta)
        self.masters = None if masters is None else list(masters)
        if not self.params:
            raise ValueError("params is empty")
        _need(self.params[0], "params[0]")
        self.device, self.dtype = self.params[0].device, self.params[0].dtype
        self.param_code = _layer_dtype(self.params[0])
        if self.masters is not None and self.dtype != torch.bfloat16:
            raise ValueError("masters go with bfloat16 params")
        lists = [("momenta", self.momenta), ("masters", self.masters)]
        for nm, lst in lists:
            if lst is not None and len(lst) != len(self.params):
                raise ValueError(f"{nm} has {len(lst)} tensors, expected {len(self.params)}")
        self.table = (_lib.DoraMuonTensor * len(self.params))()
        written = []
        for i, (e, p) in enumerate(zip(self.table, self.params)):
            _need(p, f"params[{i}]", self.dtype, None, self.device)
            if p.dim() != 2:
                raise ValueError(f"params[{i}] has {p.dim()} dimensions, expected a matrix")
            e.rows, e.cols = p.shape
            e.param = p.data_ptr()
            written.append((p, f"params[{i}]"))
            for nm, lst in lists:
                if lst is not None:
                    _need(lst[i], f"{nm}[{i}]", torch.float32, p.shape, self.device)
                    written.append((lst[i], f"{nm}[{i}]"))
            e.momentum = self.momenta[i].data_ptr()
            e.master = None if self.masters is None else self.masters[i].data_ptr()
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), nm)
                       for t, nm in written if t.numel())
        for a, b in zip(spans, spans[1:]):
            if b[0] < a[1]:
                raise ValueError(f"{a[2]} and {b[2]} share memory: a step writes both")
        self._written, self._ends = spans, [a[1] for a in spans]   # in order, and apart from each other
        flat = [v for a in spans for v in a[:2]]
        self._spans = (ctypes.c_int64 * max(len(flat), 1))(*flat)
        self._address = ctypes.addressof(self.table)
        self._bytes = {}   # of workspace, for the coefficients of the last step

    def unchanged(self):
        """Whether every tensor still has the storage it had when the plan was made."""
        masters = self.masters or [None] * len(self.params)
        return all(p.data_ptr() == (e.param or 0) and p.dtype == self.dtype
                   and p.shape == (e.rows, e.cols) and m.data_ptr() == (e.momentum or 0)
                   and (w is None or w.data_ptr() == (e.master or 0))
                   and p.is_contiguous() and m.is_contiguous() and m.shape == p.shape
                   for e, p, m, w in zip(self.table, self.params, self.momenta, masters))

    def _take_grads(self, grads, adjust):
        """Checks the gradients and notes them and their updates' factors; returns their dtype's code."""
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} params")
        if not self.unchanged():
            raise ValueError("a tensor's storage has changed since the plan was made")
        for nm, lst, dt in (("params", self.params, self.dtype), ("momenta", self.momenta, torch.float32),
                            ("masters", self.masters, torch.float32)):
            for i, (t, p) in enumerate(zip(lst or (), self.params)):
                _need(t, f"{nm}[{i}]", dt, p.shape, self.device)
        gdt = grads[0].dtype if isinstance(grads[0], torch.Tensor) else None
        if gdt is not None and gdt not in _DT:
            raise ValueError(f"unsupported dtype {gdt}; use float32 or bfloat16")
        for i, (g, p, e) in enumerate(zip(grads, self.params, self.table)):
            e.grad = _need(g, f"grads[{i}]", gdt, p.shape, self.device).data_ptr()
            e.scale = update_factor(adjust, e.rows, e.cols)
            end = g.data_ptr() + g.numel() * g.element_size()
            for lo, hi, name in self._written[bisect.bisect_right(self._ends, g.data_ptr()):]:
                if lo >= end:
                    break
                raise ValueError(f"grads[{i}] and {name} share memory: a step writes one and reads the other")
        return _DT[gdt]


def update_factor(adjust, rows, cols):
    """The factor on an orthogonalised update: "rms" 0.2 sqrt(max(rows, cols)), which gives it the
    root mean square of AdamW's; "spectral" sqrt(max(1, rows / cols)); or a number."""
    if adjust == "rms":
        return 0.2 * max(rows, cols) ** 0.5
    if adjust == "spectral":
        return max(1.0, rows / max(cols, 1)) ** 0.5
    if isinstance(adjust, str):
        raise ValueError(f"adjust is {adjust!r}, expected rms, spectral or a number")
    return float(adjust)


def dora_muon(plan, grads, *, lr, momentum=0.95, nesterov=True, weight_decay=0.0,
              coefficients=NEWTON_SCHULZ, eps=1e-7, adjust="rms", workspace=None):
    """One step with orthogonalised updates on the matrices of a plan, in place:
    m = momentum m + (1 - momentum) g, u = momentum m + (1 - momentum) g (m without ``nesterov``),
    p = p (1 - lr weight_decay) - lr update_factor(adjust) orthogonalised(u).

    ``grads``: one contiguous tensor per parameter, all bf16 or all float32, none of them over memory that
    the step writes.
    """
    grads = grads if isinstance(grads, list) else list(grads)
    factor = None if adjust == "rms" else update_factor(adjust, 1, 1)
    code = _compiled().muon_grads(plan.params, plan.momenta, plan.masters, plan._address, grads, factor,
                                  ctypes.addressof(plan._spans), len(plan._written))
    if code is None or plan.params[0].dtype != plan.dtype:
        code = plan._take_grads(grads, adjust)
    elif adjust == "spectral":
        for e in plan.table:
            e.scale = update_factor(adjust, e.rows, e.cols)
    iteration, _held = _iteration(coefficients, eps)
    how = _lib.DoraMuonOptions(iteration, plan.param_code, code, int(bool(nesterov)), 0, float(lr),
                               float(momentum), float(weight_decay))
    L, n = _lib.lib(), len(plan.params)
    if workspace is None:
        # depends on the sizes, which a plan keeps, and the coefficients; 0 where the step will be refused
        # for another option, which says nothing about the next one
        key = tuple(_held)
        nbytes = plan._bytes.get(key) or L.dora_muon_workspace_bytes(plan.table, n, ctypes.byref(how))
        plan._bytes = {key: nbytes}
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=plan.device)
    # (the parameters' versions go up: a backward pass that saved one from before is refused)
    _check(_compiled().muon_step(plan._address, plan.params, ctypes.addressof(how), workspace.data_ptr(),
                                 _given_ws(workspace, plan.device), _stream(plan.device)),
           "dora_muon_step")


def _second_moment(codes):
    if codes.dtype not in (torch.int8, torch.uint8):
        raise ValueError(f"codes have dtype {codes.dtype}, expected int8 (exp_avg) or uint8 (exp_avg_sq)")
    return codes.dtype == torch.uint8


def dora_adamw_dequantize(codes, scales, *, dtype=torch.float32):
    """The values of 8-bit states: exp_avg of int8 codes, exp_avg_sq of uint8 codes."""
    if _on_gpu(codes) and dtype in _DT:
        out = _compiled().dequantize(codes, scales, dtype == torch.bfloat16, _stream(codes.device))
        if out is not None:
            return out
    _need(codes, "codes")
    second = _second_moment(codes)
    n = codes.numel()
    _need(scales, "scales", torch.float32, (-(-n // _lib.STATE_BLOCK),), codes.device)
    if dtype not in _DT:
        raise ValueError(f"unsupported dtype {dtype}; use float32 or bfloat16")
    out = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    _check(_lib.lib().dora_adamw_dequantize(_ptr(codes), _ptr(scales), n, int(second), _ptr(out),
                                            _DT[dtype], _stream(codes.device)),
           "dora_adamw_dequantize")
    return out


def dora_adamw_quantize(values, *, second_moment):
    """8-bit codes and scales of float32 moments: (int8, float32) of exp_avg, (uint8, float32) of
    exp_avg_sq (``second_moment``)."""
    _need(values, "values", torch.float32)
    n, dev = values.numel(), values.device
    codes = torch.empty(values.shape, dtype=torch.uint8 if second_moment else torch.int8, device=dev)
    scales = torch.empty(-(-n // _lib.STATE_BLOCK), dtype=torch.float32, device=dev)
    _check(_lib.lib().dora_adamw_quantize(_ptr(values), n, int(bool(second_moment)), _ptr(codes),
                                          _ptr(scales), _stream(dev)), "dora_adamw_quantize")
    return codes, scales


def timing_enable(on: bool = True):
    _lib.lib().dora_timing_enable(1 if on else 0)


def timing_collect() -> dict:
    """{kernel label: (launch count, total ms)} since the last collect."""
    buf = ctypes.create_string_buffer(1 << 16)
    rc = _lib.lib().dora_timing_collect(buf, len(buf))
    if rc < 0:
        raise DoraError(rc, "dora_timing_collect")
    return {k: (int(v[0]), float(v[1])) for k, v in json.loads(buf.value.decode()).items()}


def probe_mfma(iters: int, blocks: int, *, out=None):
    """Launch the sustained-MFMA probe on the current stream; returns (out, flops)."""
    import torch
    if out is None:
        out = torch.empty(blocks * 256, dtype=torch.float32, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    L = _lib.lib()
    rc = L.dora_probe_mfma(int(iters), int(blocks), out.data_ptr(), st)
    if rc != 0:
        raise DoraError(rc, "dora_probe_mfma")
    return out, L.dora_probe_mfma_flops(int(iters), int(blocks))


def probe_stream(a, b, c):
    """c = a + b over float32 tensors on the current stream (HBM streaming probe)."""
    import torch
    for t in (a, b, c):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != a.numel():
            raise ValueError("probe_stream takes three contiguous float32 tensors of one size")
    st = torch.cuda.current_stream().cuda_stream
    rc = _lib.lib().dora_probe_stream(a.data_ptr(), b.data_ptr(), c.data_ptr(), a.numel() * 4, st)
    if rc != 0:
        raise DoraError(rc, "dora_probe_stream")
    return c

