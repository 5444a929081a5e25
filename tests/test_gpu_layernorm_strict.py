"""Layer norm once more, against the same bars but with comparisons that a NaN fails too, and the
weight's gradient where offsets pass 32 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import test_gpu_layernorm as base

pytestmark = pytest.mark.gpu
ops = base.ops
U = base.U
WIDE = [(3, 8200), (300, 9001), (7, 10240), (5, 10241), (261, 12289), (2, 14336), (6, 14337),
        (300, 16383), (520, 16384), (4, 16385)]


def held(got, want, bar, what):
    bad = ~(np.abs(got - want) <= bar)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", base.SIZES + WIDE)
def test_no_output_is_nan(ops, rows, width, dtype, monkeypatch):
    monkeypatch.setattr(base, "held", held)
    base.test_forward_and_backward(ops, rows, width, dtype)


@pytest.mark.parametrize("rows,width", [(263000, 8192), ((1 << 21) + 77, 24)])
def test_weight_gradient_past_32_bits(ops, rows, width):
    """Chains of at most rows / 256 + 300 float32 additions, xhat's own roundings (4 of |x| + |mean|
    in units of 1 / rstd), half a last place of bf16."""
    base.say("layernorm", rows, width)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x, gy = (torch.empty(rows, width, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    step = 1 << 14
    for t in (x, gy):
        for r in range(0, rows, step):
            t[r:r + step] = torch.randn(t[r:r + step].shape, device="cuda", generator=gen)
    _, mean, rstd = ops.dora_layernorm(x, None, None)
    _, gw, gb = ops.dora_layernorm_backward(gy, x, None, mean, rstd, need=("weight", "bias"))
    want, terms, carry, wantb, termsb = (torch.zeros(width, dtype=torch.float64, device="cuda")
                                         for _ in range(5))
    for r in range(0, rows, step):
        g, v = gy[r:r + step].double(), x[r:r + step].double()
        mu, rs = mean[r:r + step].double()[:, None], rstd[r:r + step].double()[:, None]
        n = (v - mu) * rs
        want += (g * n).sum(0)
        terms += (g * n).abs().sum(0)
        carry += (g.abs() * (v.abs() + mu.abs()) * rs).sum(0)
        wantb += g.sum(0)
        termsb += g.abs().sum(0)
    N = rows / 256 + 300
    assert ((gw.double() - want).abs() <= U * (N * terms + 4 * carry) + want.abs() * 2.0 ** -8).all()
    assert ((gb.double() - wantb).abs() <= U * N * termsb + wantb.abs() * 2.0 ** -8).all()
    del x, gy
    torch.cuda.empty_cache()
