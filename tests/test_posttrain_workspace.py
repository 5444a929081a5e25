"""The workspaces of orthogonalised matrices and Muon steps: bytes an element as the header says, by how
often S is formed anew on the way."""
from __future__ import annotations

import ctypes
import os

import pytest

from parameter_efficient_fine_dora_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libdora.so not built")
USUAL = (3.4445, -4.7750, 2.0315)
MOST = {"bf16": 65536.0, "f32": 20.0, "param": 1024.0}   # the factor on S's rounding up to which it is kept


def anew(coefficients, most):
    """How often S is formed anew: where sum |b / a| prod a^2 of the steps since would pass `most`."""
    times, grown, gain = 0, 0.0, 1.0
    for k, (a, b, _) in enumerate(coefficients):
        if k and grown + abs(b / a) * gain > most:
            times, grown, gain = times + 1, 0.0, 1.0
        grown += abs(b / a) * gain
        gain *= a * a
    return times


def iteration(steps):
    flat = (ctypes.c_double * (3 * steps))(*(USUAL * steps))
    return _lib.DoraNewtonSchulz(ctypes.addressof(flat), steps, 0, 1e-7), flat


def orthogonalize(rows, cols, dtype, steps):
    z, held = iteration(steps)
    o = _lib.DoraOrthogonalizeOptions(z, dtype, 0)
    t = (_lib.DoraMatrix * 1)(_lib.DoraMatrix(None, None, rows, cols))
    return _lib.lib().dora_orthogonalize_workspace_bytes(t, 1, ctypes.byref(o))


def muon(rows, cols, dtype, master, steps):
    z, held = iteration(steps)
    o = _lib.DoraMuonOptions(z, dtype, _lib.BF16, 1, 0, 1e-3, 0.95, 0.0)
    t = (_lib.DoraMuonTensor * 1)(_lib.DoraMuonTensor(None, None, None, 0x10000 if master else None, rows, cols, 1.0))
    return _lib.lib().dora_muon_workspace_bytes(t, 1, ctypes.byref(o))


def element(got, n, m):
    """Bytes an element beside 20 n^2, without partial sums: a fifth of a byte at these lengths."""
    value = (got - 20 * n * n) / (n * m)
    assert 0 <= value % 1 < 0.2, value
    return int(value)


@pytest.mark.parametrize("steps", range(1, 17))
@pytest.mark.parametrize("n,m", [(64, 1 << 17), (256, 1 << 18)])
def test_bytes_an_element(steps, n, m):
    coefficients = (USUAL,) * steps

    def pairs(times):    # float32 matrices, and updates
        return 4 if times == 0 or (n <= 64 and times <= 2) else 8

    for rows, cols in ((n, m), (m, n)):
        times = anew(coefficients, MOST["bf16"])
        assert element(orthogonalize(rows, cols, _lib.BF16, steps), n, m) == (2, 6, 8)[min(times, 2)]
        assert element(muon(rows, cols, _lib.BF16, False, steps), n, m) == pairs(times)
        assert element(orthogonalize(rows, cols, _lib.F32, steps), n, m) == pairs(anew(coefficients, MOST["f32"]))
        times = anew(coefficients, MOST["param"])
        assert element(muon(rows, cols, _lib.F32, False, steps), n, m) == pairs(times)
        assert element(muon(rows, cols, _lib.BF16, True, steps), n, m) == pairs(times)


def test_the_usual_iteration():
    assert [anew((USUAL,) * 5, v) for v in MOST.values()] == [0, 2, 1]
    assert [anew((USUAL,) * 10, v) for v in MOST.values()] == [1, 4, 3]


def test_sides_are_padded():
    """n to 128, or to 64 where that holds it; m to 128."""
    def padded(v, to):
        return -(-v // to) * to

    for n, m in ((1, 129), (63, 1000), (65, 1000), (129, 3333)):
        nt, mt = padded(n, 64 if n <= 64 else 128), padded(m, 128)
        got = orthogonalize(n, m, _lib.BF16, 5)
        parts = 32 * 4 * nt * nt + 4096
        assert 2 * nt * mt + 20 * nt * nt <= got <= 2 * nt * mt + 20 * nt * nt + parts
