"""Weight decay whose factor 1 - lr weight_decay is no float32 number."""
from __future__ import annotations

import numpy as np
import pytest
import torch

LR, DECAY = 0.01, 0.23   # 1 - 0.0023, of which float32 loses more than 2^-26
N = (512, 2048)


def parameters():
    rng = np.random.default_rng(1)
    return rng.uniform(0.5, 1.0, N).astype(np.float32)


def mean_error(got, p):
    return float((got.astype(np.float64) - p.astype(np.float64) * (1.0 - LR * DECAY)).mean())


def test_the_plain_float32_factor_is_off():
    """What the step's second term is for: without it 2^20 parameters are off by p times the factor's
    rounding on average, where their own roundings, up to 2^-25 either way, average out to some 2^-35."""
    p = parameters()
    factor = np.float32(1.0 - LR * DECAY)
    lost = float(factor) - (1.0 - LR * DECAY)
    assert abs(lost) > 2.0 ** -26
    plain = (p.astype(np.float64) * float(factor)).astype(np.float32)   # one rounding
    assert abs(mean_error(plain, p)) > 0.7 * abs(lost) > 8 * 2.0 ** -30


@pytest.mark.gpu
@pytest.mark.parametrize("master", [False, True])
def test_the_factors_rounding_does_not_add_up(master):
    from parameter_efficient_fine_dora_amd import ops
    p = parameters()
    w = torch.from_numpy(p).cuda()
    zero = torch.zeros(N, device="cuda")
    param = w.bfloat16() if master else w
    plan = ops.MuonPlan([param], [torch.zeros(N, device="cuda")], masters=[w] if master else None)
    ops.dora_muon(plan, [zero], lr=LR, weight_decay=DECAY)    # (an update of zero)
    got = w.cpu().numpy()
    want = p.astype(np.float64) * (1.0 - LR * DECAY)
    # the result's rounding, and the small term's, 2^-24 of 2^-25
    assert np.abs(got - want).max() <= 2.0 ** -25 * (1 + 2.0 ** -20)
    assert abs(mean_error(got, p)) <= 2.0 ** -30
    if master:
        assert torch.equal(param, w.bfloat16())
