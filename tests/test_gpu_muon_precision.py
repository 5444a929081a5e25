"""Muon's updates of bf16 parameters, with and without masters: any magnitude, and 22 bits of the update."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import posttrain as oracle

pytestmark = pytest.mark.gpu
STEPS = ((3.4445, -4.7750, 2.0315),) * 5


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from parameter_efficient_fine_dora_amd import _lib, ops
    _lib.lib()
    return ops


def host(t):
    return t.detach().double().cpu().numpy()


def step(ops, g, master=False, **how):
    """What a step without momentum makes of a bf16 parameter of zeros (or of its master): minus X(g)."""
    p, m = torch.zeros(g.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(g.shape, device="cuda")
    w = torch.zeros(g.shape, device="cuda") if master else None
    plan = ops.MuonPlan([p], [m], masters=[w] if master else None)
    ops.dora_muon(plan, [g], lr=1.0, momentum=0.0, adjust=1.0, **how)
    assert torch.equal(m, g.float())
    return w if master else p


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("size", [(24, 80), (80, 24), (64, 300), (130, 140), (300, 90)], ids=str)
@pytest.mark.parametrize("eps", [1e-7, 2.0 ** -41, 2.0 ** -100])
def test_any_magnitude(ops, size, eps, master):
    """Well conditioned gradients: no direction is raised by more than the iteration raises it, so half a step
    of the result and a thousandth of that decide.  1e33 of 12000 elements is within bf16's range."""
    g = torch.randn(*size, generator=torch.Generator().manual_seed(1))
    for scale in (1e-12, 1e-3, 1.0, 16.0, 1e4, 1e10, 1e19, 1e25, 1e33):
        x = (g * scale).bfloat16().cuda()
        got = host(step(ops, x, master, eps=eps))
        want = -oracle.orthogonalize(host(x), STEPS, eps)
        half = 2.0 ** -8 if not master else 2.0 ** -10
        assert np.linalg.norm(got - want) <= half * np.linalg.norm(want), (scale, np.linalg.norm(got - want))


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("size", [(24, 80), (80, 24), (64, 300), (130, 140), (300, 90)], ids=str)
def test_a_weak_direction_under_a_strong_one(ops, size, master):
    """X - S X takes the one strong direction away and leaves the rest, 2^-14 of it.  The update's halves lose
    2^-22 of the strong one's elements, S as much, twice; X - S X passes what is lost on with a slope of at
    most 2: 6 2^-22 in norm, and half a step of the result."""
    gen = torch.Generator().manual_seed(2)
    u, v = torch.randn(size[0], 1, generator=gen), torch.randn(1, size[1], generator=gen)
    strong, weak = u @ v, torch.randn(*size, generator=gen)
    g = (strong / strong.norm() + 2.0 ** -14 * weak / weak.norm()).cuda()
    coefficients = ((1.0, -1.0, 0.0),)
    got = host(step(ops, g, master, coefficients=coefficients))
    want = -oracle.orthogonalize(host(g), coefficients, 1e-7)
    half = 2.0 ** -8 if not master else 2.0 ** -24
    off = np.linalg.norm(got - want)
    assert off <= 6 * 2.0 ** -22 + half * np.linalg.norm(want), (off * 2.0 ** 22, np.linalg.norm(want))
