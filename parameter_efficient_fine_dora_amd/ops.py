"""Thin torch binding of libdora.so: same names as the C ABI.

Only argument marshalling happens here: tensors are checked for device,
dtype, shape and contiguity, output and workspace buffers are allocated by
torch's caching allocator (the library allocates nothing), and the raw device
pointers plus torch's current HIP stream are passed to the library.  Every
step of the computation runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
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
            "dora_adamw_dequantize")))
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

