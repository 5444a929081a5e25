"""The policy loss of tokens whose probabilities lie far apart: ratios and divergences at float64's end,
beyond it and infinite, each against the definition."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
INF = math.inf
FAR = [709.5, 709.75, 710.0, 800.0, 800.3, 1000.0, 1000.3, 1099.9, 1e5, 3e38, INF]
HIGH, LOW = 0.28, 0.2


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from parameter_efficient_fine_dora_amd import _lib, ops
    _lib.lib()
    return ops


def exp(x):
    return math.exp(x) if x < 709.78 else INF


def definition(x, a, dual, d, kl_coef):
    """(loss, slope, kl, held, ratio) of one token with logp - old = x and ref - logp = d."""
    ratio = exp(x)
    if a >= 0:
        held, gain = a > 0 and ratio > 1 + HIGH, a * min(ratio, 1 + HIGH)
        flat = ratio > 1 + HIGH
    else:
        held = flat = ratio < 1 - LOW or ratio > dual
        gain = a * min(max(ratio, 1 - LOW), dual)
    slope = 0.0 if flat else -a * ratio
    kl = 0.0
    if d is not None:
        e = INF if d > 709.78 else math.expm1(d)
        kl = INF if abs(d) == INF else e - d
        gain, slope = gain - kl_coef * kl, slope - kl_coef * e
    return -gain, slope, kl, float(held), ratio


def same(got, want):
    """A float32 rounding: half of 2^-149 where numbers lie that far apart, infinite beyond the largest."""
    want = math.copysign(INF, want) if abs(want) > 3.4028236e38 else want
    return got == want or abs(got - want) <= 2.0 ** -24 * (1 + 1e-6) * abs(want) + 2.0 ** -150


def one(value):
    return torch.full((1, 1), value, device="cuda")


@pytest.mark.parametrize("sign", [1, -1], ids=["above", "below"])
@pytest.mark.parametrize("advantage", [1.5, -1.5, 0.0])
@pytest.mark.parametrize("dual", [None, 3.0])
@pytest.mark.parametrize("reduce", ["token", "sequence"])
def test_ratios(ops, sign, advantage, dual, reduce):
    for x in FAR:
        logp, old = one(-0.25), one(-0.25 - sign * x)
        adv = torch.full((1,), advantage, device="cuda")
        how = dict(clip=(LOW, HIGH), dual_clip=dual, reduce=reduce)
        x = float(logp.double() - old.double())
        loss, stats, weight = ops.dora_policy_loss(logp, old, adv, **how)
        grad = ops.dora_policy_loss_backward(torch.ones((), device="cuda"), weight, logp, old, adv, **how)
        want = definition(x, advantage, dual or INF, None, 0.0)
        assert same(float(loss), want[0]) and same(float(grad), want[1]), (x, float(loss), float(grad), want)
        assert stats.tolist()[1] == want[3] and same(float(stats[2]), want[4]), (x, stats.tolist(), want)


@pytest.mark.parametrize("sign", [1, -1], ids=["above", "below"])
@pytest.mark.parametrize("kl_coef", [0.0, 0.5])
def test_divergences(ops, sign, kl_coef):
    for d in FAR:
        logp, ref = one(-0.25), one(-0.25 + sign * d)
        adv = torch.full((1,), 0.5, device="cuda")
        d = float(ref.double() - logp.double())
        how = dict(clip=(LOW, HIGH), ref_logp=ref, kl_coef=kl_coef)
        loss, stats, weight = ops.dora_policy_loss(logp, logp, adv, **how)
        grad = ops.dora_policy_loss_backward(torch.ones((), device="cuda"), weight, logp, logp, adv, **how)
        want = definition(0.0, 0.5, INF, d if kl_coef else None, kl_coef)
        assert same(float(loss), want[0]) and same(float(grad), want[1]), (d, float(loss), float(grad), want)
        assert same(float(stats[0]), definition(0.0, 0.5, INF, d, 0.5)[2]), (d, stats.tolist())


def test_a_token_without_probability(ops):
    """logp of -infinity: the ratio is 0, the divergence and its slope infinite; the other sequences' tokens
    and the token sums' other terms are as without it."""
    logp = torch.tensor([[-0.5, -1.0], [-0.25, -2.0]], device="cuda")
    old, ref = logp - 0.125, logp + 0.25
    adv = torch.tensor([1.0, -1.0], device="cuda")
    logp[0, 1] = -INF
    how = dict(clip=(LOW, HIGH), ref_logp=ref, kl_coef=0.1, reduce="sequence")
    loss, stats, weight = ops.dora_policy_loss(logp, old, adv, **how)
    grad = ops.dora_policy_loss_backward(torch.ones((), device="cuda"), weight, logp, old, adv, **how)
    assert float(loss) == INF and float(stats[0]) == INF and float(stats[3]) == 4.0
    assert same(float(stats[2]), 3 * math.exp(0.125) / 4) and float(grad[0, 1]) == -INF
    for i, j in ((0, 0), (1, 0), (1, 1)):
        want = definition(0.125, float(adv[i]), INF, 0.25, 0.1)[1] * 0.25
        assert abs(float(grad[i, j]) - want) <= 2.0 ** -23 * abs(want)
