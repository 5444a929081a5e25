"""Advantages of a packed batch that has as many tokens as sequences: the shape says nothing, the caller does."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import posttrain as oracle

pytestmark = pytest.mark.gpu
LENGTHS = [0, 3, 1, 0, 0, 2]          # six sequences of six tokens
HALF = 2.0 ** -24 * (1 + 1e-6)


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from parameter_efficient_fine_dora_amd import _lib, ops
    _lib.lib()
    return ops


def batch(seed=0):
    rng = np.random.default_rng(seed)
    offsets = np.concatenate([[0], np.cumsum(LENGTHS)]).astype(np.int64)
    logp = -rng.random(6).astype(np.float32)
    old = (logp + 0.3 * rng.standard_normal(6)).astype(np.float32)
    return logp, old, rng.standard_normal(6).astype(np.float32), offsets


def dev(a):
    return torch.from_numpy(a).cuda()


@pytest.mark.parametrize("reduce", ["token", "sequence"])
@pytest.mark.parametrize("per_sequence", [None, False, True])
@pytest.mark.parametrize("checked", [False, True], ids=["compiled", "checked"])
def test_as_many_tokens_as_sequences(ops, reduce, per_sequence, checked):
    logp, old, adv, offsets = batch()
    where = oracle.spans((6,), offsets)
    each = np.repeat(adv, LENGTHS) if per_sequence else adv
    value, stats, weight, grad = oracle.policy_loss(logp, old, each, where, None, None, reduce=reduce)
    how = dict(offsets=dev(offsets), reduce=reduce, per_sequence=per_sequence)
    room = dict(workspace=torch.empty(1 << 16, dtype=torch.uint8, device="cuda")) if checked else {}
    loss, _, w = ops.dora_policy_loss(dev(logp), dev(old), dev(adv), **how, **room)
    out = dict(grad_logp=torch.empty(6, device="cuda")) if checked else {}
    got = ops.dora_policy_loss_backward(torch.ones((), device="cuda"), w, dev(logp), dev(old), dev(adv), **how, **out)
    # one rounding of the value; two of a gradient, whose weight is rounded too
    assert abs(float(loss) - value) <= HALF * abs(value) + 1e-15
    assert (np.abs(got.double().cpu().numpy() - grad) <= 2 * HALF * np.abs(grad)).all()


def test_through_autograd_and_what_is_refused(ops):
    from parameter_efficient_fine_dora_amd.module import policy_loss
    logp, old, adv, offsets = batch(1)
    x = dev(logp).requires_grad_()
    loss, _ = policy_loss(x, dev(old), dev(adv), offsets=dev(offsets), per_sequence=True)
    loss.backward()
    *_, grad = oracle.policy_loss(logp, old, np.repeat(adv, LENGTHS), oracle.spans((6,), offsets), None, None)
    assert (np.abs(x.grad.double().cpu().numpy() - grad) <= 2 * HALF * np.abs(grad)).all()
    l = torch.zeros(4, 6, device="cuda")
    for per_sequence, shape in ((True, (4, 6)), (False, (4,))):
        with pytest.raises(ValueError, match="advantages has shape"):
            ops.dora_policy_loss(l, l, torch.zeros(shape, device="cuda"), per_sequence=per_sequence)
        with pytest.raises(ValueError, match="advantages has shape"):
            ops.dora_policy_loss_backward(torch.ones((), device="cuda"), torch.ones(1, device="cuda"), l, l,
                                          torch.zeros(shape, device="cuda"), per_sequence=per_sequence)
