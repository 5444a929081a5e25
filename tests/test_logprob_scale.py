"""Scales of the token log probabilities at the C boundary, on the host: those whose product with
log2(e) float32 cannot hold are refused before anything is enqueued."""
from __future__ import annotations

import ctypes
import os

import pytest

from parameter_efficient_fine_dora_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libdora.so not built")


@pytest.mark.parametrize("scale,taken", [
    (2.0 ** 127, False), (2.4e38, False), (3.4e38, False), (float("inf"), False), (float("nan"), False),
    (0.0, False), (-1.0, False), (1.7e38, True), (1.0, True), (1e-45, True)])
def test_scales(scale, taken):
    L = _lib.lib()
    s = _lib.DoraLogprobShape(0, 8, 8, _lib.F32, 0, scale, 0)     # no rows: nothing is enqueued
    want = 0 if taken else _lib.ERR_CODE["DORA_ERR_FLAGS"]
    assert L.dora_token_logprob_forward(ctypes.byref(s), *([None] * 8), 0, None) == want
    assert L.dora_token_logprob_backward(ctypes.byref(s), *([None] * 7), None) == want
