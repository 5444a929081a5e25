"""The preference gradient of short sequences and many pairs: on both sides of the rules that choose between
one launch and two, against the definition."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import posttrain as oracle

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24 * (1 + 1e-6)


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from parameter_efficient_fine_dora_amd import _lib, ops
    _lib.lib()
    return ops


# sequences, tokens of each, pairs: 64 pairs are a look, 256 tokens a round; eight looks are the border
SIZES = [(1, 1, 1), (8, 31, 4), (8, 32, 4), (8, 33, 4), (40, 63, 128), (40, 64, 128), (40, 65, 128), (40, 64, 129),
         (20, 127, 256), (20, 128, 256), (20, 129, 256), (20, 129, 257), (512, 1, 256), (512, 8, 200), (700, 3, 65)]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("packed", [False, True], ids=["padded", "packed"])
def test_gradient(ops, size, packed):
    S, L, P = size
    rng = np.random.default_rng(S + L + P)
    n = S * L
    if packed:   # the same tokens in sequences of other lengths, empty ones among them
        cuts = np.sort(rng.integers(0, n + 1, S - 1))
        offsets, shape = np.concatenate([[0], cuts, [n]]).astype(np.int64), (n,)
    else:
        offsets, shape = None, (S, L)
    where = oracle.spans(shape, offsets)
    chosen, rejected = rng.integers(0, S, (2, P))
    logit, g = (rng.standard_normal(P).astype(np.float32) for _ in range(2))
    count = np.array([b - a for a, b in where], np.float32)
    live = rng.random(n) < 0.8

    def dev(a):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()

    for normalize in (False, True):
        got = ops.dora_preference_loss_backward(dev(g), dev(logit), dev(count), dev(chosen), dev(rejected),
                                                shape=shape, mask=dev(live.reshape(shape)), offsets=dev(offsets),
                                                normalize=normalize)
        want = oracle.preference_backward(g, logit, count, chosen, rejected, where, n, live, normalize=normalize)
        # the sum of a sequence's pairs is float64, and rounded once
        off = np.abs(got.double().cpu().numpy().reshape(-1) - want)
        assert (off <= HALF * np.abs(want) + 1e-12 * np.abs(g).sum()).all(), off.max()
