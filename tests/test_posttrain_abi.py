"""Preference loss, policy loss and orthogonalised updates at the C boundary, on the host: structs
as the header lays them out, arguments refused before anything is enqueued, workspace sizes."""
import ctypes
import os
import re

import pytest

from parameter_efficient_fine_dora_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libdora.so not built")
E = _lib.ERR_CODE
FAKE = 0x10000   # never dereferenced: every call here is refused
HUGE = 1 << 40
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "dora_posttrain.h")


def test_library_exports_and_binds_every_declared_symbol():
    names = re.findall(r"DORA_API\s+[\w\s\*]+?\b(dora_\w+)\s*\(", open(HEADER).read())
    assert len(names) == len(set(names)) >= 6
    for name in names:
        assert hasattr(_lib.lib(), name) and name in _lib._SIGS, name


def test_structs_and_numbers_are_the_headers():
    assert ctypes.sizeof(_lib.DoraTokenBatch) == 40
    assert ctypes.sizeof(_lib.DoraPreferenceOptions) == 32
    assert _lib.DoraPreferenceOptions.beta.offset == 8
    assert ctypes.sizeof(_lib.DoraPolicyOptions) == 48
    assert _lib.DoraPolicyOptions.reduce.offset == 40
    text = open(HEADER).read()
    for prefix, table in (("DORA_PREFERENCE_", _lib.PREFERENCE_KIND), ("DORA_REDUCE_", _lib.POLICY_REDUCE)):
        found = {k.lower(): int(v) for k, v in re.findall(prefix + r"(\w+)\s*=\s*(\d+)", text)}
        assert found == table


def batch(tokens=40, sequences=4, length=10, offsets=None, mask=None):
    return _lib.DoraTokenBatch(tokens, sequences, length, offsets, mask)


def pref(kind=0, normalize=0, beta=0.1, margin=0.0, smoothing=0.0):
    return _lib.DoraPreferenceOptions(kind, normalize, beta, margin, smoothing)


def policy(low=0.2, high=0.2, dual=float("inf"), kl=0.0, by=0.0, reduce=0, per=0):
    return _lib.DoraPolicyOptions(low, high, dual, kl, by, reduce, per)


def pref_forward(b=None, o=None, pairs=2, args=None, ws=FAKE, nb=HUGE):
    b, o = b or batch(), o or pref()
    return _lib.lib().dora_preference_forward(ctypes.byref(b), ctypes.byref(o), pairs,
                                              *(args or [FAKE] * 8), ws, nb, None)


def pref_backward(b=None, o=None, pairs=2, args=None, ws=FAKE, nb=HUGE):
    b, o = b or batch(), o or pref()
    return _lib.lib().dora_preference_backward(ctypes.byref(b), ctypes.byref(o), pairs,
                                               *(args or [FAKE] * 6), ws, nb, None)


def policy_forward(b=None, o=None, args=None, ws=FAKE, nb=HUGE):
    b, o = b or batch(), o or policy()
    return _lib.lib().dora_policy_forward(ctypes.byref(b), ctypes.byref(o), *(args or [FAKE] * 7), ws,
                                          nb, None)


def policy_backward(b=None, o=None, args=None):
    b, o = b or batch(), o or policy()
    return _lib.lib().dora_policy_backward(ctypes.byref(b), ctypes.byref(o), *(args or [FAKE] * 7), None)


EVERY = (pref_forward, pref_backward, policy_forward, policy_backward)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), "DORA_ERR_SHAPE"), (dict(sequences=-1), "DORA_ERR_SHAPE"),
    (dict(tokens=1 << 34, sequences=1, length=1 << 34), "DORA_ERR_SHAPE"),
    (dict(tokens=1 << 31, sequences=1 << 31, length=1), "DORA_ERR_SHAPE"),
    (dict(length=11), "DORA_ERR_SHAPE"), (dict(tokens=41), "DORA_ERR_SHAPE"),
    (dict(sequences=0), "DORA_ERR_SHAPE"), (dict(offsets=FAKE), "DORA_ERR_SHAPE"),
    (dict(length=0, offsets=FAKE + 4), "DORA_ERR_ALIGN"),
])
def test_batches_refused(kw, code):
    b = batch(**kw)
    for call in EVERY:
        assert call(b=b) == E[code], call
    assert _lib.lib().dora_preference_workspace_bytes(ctypes.byref(b)) == 0
    assert _lib.lib().dora_policy_workspace_bytes(ctypes.byref(b), ctypes.byref(policy())) == 0


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw", [dict(kind=-1), dict(kind=3), dict(normalize=2), dict(beta=0.0),
                                dict(beta=-1.0), dict(beta=NAN), dict(beta=INF), dict(margin=INF),
                                dict(margin=NAN), dict(smoothing=-0.1), dict(smoothing=1.1),
                                dict(smoothing=NAN)])
def test_preference_options_refused(kw):
    for call in (pref_forward, pref_backward):
        assert call(o=pref(**kw)) == E["DORA_ERR_FLAGS"]


@pytest.mark.parametrize("kw", [dict(low=-0.1), dict(low=1.1), dict(low=NAN), dict(high=-0.1),
                                dict(high=NAN), dict(dual=0.9), dict(dual=NAN), dict(kl=-1.0),
                                dict(kl=INF), dict(kl=NAN), dict(by=-1.0), dict(by=INF), dict(reduce=2),
                                dict(reduce=-1), dict(per=2)])
def test_policy_options_refused(kw):
    for call in (policy_forward, policy_backward):
        assert call(o=policy(**kw)) == E["DORA_ERR_FLAGS"]
    assert _lib.lib().dora_policy_workspace_bytes(ctypes.byref(batch()), ctypes.byref(policy(**kw))) == 0


@pytest.mark.parametrize("call,count,optional", [(pref_forward, 8, {1}), (pref_backward, 6, {2}),
                                                 (policy_forward, 7, {2}), (policy_backward, 7, {4})])
def test_pointers_refused(call, count, optional):
    for i in range(count):
        for bad, code in ((None, "DORA_ERR_NULL"), (FAKE + 2, "DORA_ERR_ALIGN")):
            if bad is None and i in optional:   # (count is not read without normalize)
                continue
            args = [FAKE] * count
            args[i] = bad
            assert call(args=args) == E[code], (i, bad)
    assert pref_backward(o=pref(normalize=1), args=[FAKE, FAKE, None, FAKE, FAKE, FAKE]) == E["DORA_ERR_NULL"]


def test_null_structs_and_pairs_refused():
    L = _lib.lib()
    b, o, p = batch(), pref(), policy()
    assert L.dora_preference_forward(None, ctypes.byref(o), 1, *[FAKE] * 8, FAKE, HUGE, None) == E["DORA_ERR_NULL"]
    assert L.dora_preference_forward(ctypes.byref(b), None, 1, *[FAKE] * 8, FAKE, HUGE, None) == E["DORA_ERR_NULL"]
    assert L.dora_policy_forward(ctypes.byref(b), None, *[FAKE] * 7, FAKE, HUGE, None) == E["DORA_ERR_NULL"]
    assert L.dora_policy_backward(None, ctypes.byref(p), *[FAKE] * 7, None) == E["DORA_ERR_NULL"]
    for call in (pref_forward, pref_backward):
        assert call(pairs=-1) == E["DORA_ERR_SHAPE"] and call(pairs=1 << 31) == E["DORA_ERR_SHAPE"]


def test_workspaces():
    L, b = _lib.lib(), batch()
    need = L.dora_preference_workspace_bytes(ctypes.byref(b))
    for call in (pref_forward, pref_backward):
        assert call(nb=need - 1) == E["DORA_ERR_WORKSPACE"] and call(ws=None) == E["DORA_ERR_NULL"]
        assert call(ws=FAKE + 8) == E["DORA_ERR_ALIGN"]
    for o in (policy(), policy(reduce=1)):
        need = L.dora_policy_workspace_bytes(ctypes.byref(b), ctypes.byref(o))
        assert policy_forward(o=o, nb=need - 1) == E["DORA_ERR_WORKSPACE"]
        assert policy_forward(o=o, ws=None) == E["DORA_ERR_NULL"]
    # a few numbers for every 256 tokens, and per sequence; no more for a thousand times the tokens
    # past a million
    big = batch(1 << 30, 1 << 10, 1 << 20)
    assert L.dora_preference_workspace_bytes(ctypes.byref(big)) <= 4096 * 32 + 1024 * 16
    # nothing to do: no tokens, no gradient
    assert pref_backward(b=batch(0, 0, 0), pairs=0, args=[None] * 6, ws=None, nb=0) == 0
    assert policy_backward(b=batch(0, 3, 0), args=[None] * 7) == 0
    assert pref_forward(b=batch(0, 0, 0), pairs=0, args=[None] * 8, ws=None, nb=0) == 0
