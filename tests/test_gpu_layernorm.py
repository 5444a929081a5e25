"""Layer norm forward and backward against float64.

Bars.  With u = 2^-24 and N the longest chain of float32 roundings an output can go through, an
output is held to N u times the sum of the magnitudes of its terms, and a bf16 output to half a
unit in its last place (8 significant bits: up to 2^-8 relative) more.  A row's sums are chains of at most width / 256 + 32
additions, the weight's gradient one of at most rows + 300.  The statistics handed to the backward
are the float64 ones rounded to float32."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import finetune as ref
from tests.gpu_util import download

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from parameter_efficient_fine_dora_amd import ops as _ops, _lib
    _lib.lib()
    return _ops


def say(*a):
    print(*a, flush=True)


def stored(a, dt):
    """A float64 array rounded to the dtype, on the GPU."""
    return torch.from_numpy(np.asarray(a, np.float32)).to(dt).cuda()


def half_ulp(dt, a):
    return np.abs(a) * (2.0 ** -8 if dt == torch.bfloat16 else U)


def held(got, want, bar, what):
    bad = np.abs(got - want) > bar
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got - want) - bar)))


def make(rows, width, dt, seed, bias, strided):
    rng = np.random.default_rng(seed)
    pad = 3 if strided else 0
    big = rng.standard_normal((rows, width + pad)) + rng.standard_normal((rows, 1))
    big[:, ::max(1, width // 3)] *= 15.0
    x = stored(big, dt)[:, pad // 2:pad // 2 + width]
    gy = stored(rng.standard_normal((rows, width + pad)), dt)[:, :width]
    w = stored(1 + 0.3 * rng.standard_normal(width), dt)
    b = stored(rng.standard_normal(width), dt) if bias else None
    return x, gy, w, b


SIZES = [(1, 1), (3, 2), (1, 8), (5, 7), (64, 64), (37, 100), (2, 513), (33, 1024), (130, 1031),
         (9, 2048), (300, 2056), (17, 4095), (6, 5121), (70, 8192), (5, 8193), (4, 16384),
         (3, 27648), (2, 32769), (2, 70001), (1031, 264), (2100, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", SIZES)
def test_forward_and_backward(ops, rows, width, dtype):
    say("layernorm", rows, width, dtype)
    dt = DT[dtype]
    for bias, strided in ((True, False), (False, True)):
        x, gy, w, b = make(rows, width, dt, rows * 7 + width, bias, strided)
        X, GY, W = download(x), download(gy), download(w)
        B = download(b) if bias else None
        eps = 1e-5
        Y, mean, rstd = ref.layernorm(X, W, B, eps)
        guard = torch.full((rows * width + 16,), 7.0, dtype=dt, device="cuda")
        y, mu, rs = ops.dora_layernorm(x, w, b, eps=eps,
                                       y=guard[8:8 + rows * width].view(rows, width))
        N = width / 256 + 32
        c = np.abs(X - mean[:, None])
        # the mean is off by N u mean|x|, which a constant row's spread of 0 would multiply by
        # rstd: both enter through |x - mean| + mean|x|
        off = c + np.abs(X).mean(axis=1, keepdims=True)
        term = off * rstd[:, None] * np.abs(W)
        held(download(mu), mean, N * U * np.abs(X).mean(axis=1), "mean")
        shift = N * U * np.abs(X).mean(axis=1) * rstd     # the mean's error, in units of 1 / rstd
        held(download(rs), rstd, (N * U * 2 + shift ** 2) * rstd, "rstd")
        bar = N * U * 3 * (term + (np.abs(B) if bias else 0)) + half_ulp(dt, Y)
        held(download(y), Y, bar, "y")
        assert (guard[:8] == 7).all() and (guard[8 + rows * width:] == 7).all()

        mean32, rstd32 = mean.astype(np.float32), rstd.astype(np.float32)
        GX, GW, GB = ref.layernorm_backward(GY, X, W, mean32.astype(np.float64),
                                            rstd32.astype(np.float64))
        need = ("x", "weight", "bias") if bias else ("x", "weight")
        gx, gw, gb = ops.dora_layernorm_backward(gy, x, w, torch.from_numpy(mean32).cuda(),
                                                 torch.from_numpy(rstd32).cuda(), need=need)
        xhat = (X - mean32[:, None].astype(np.float64)) * rstd32[:, None]
        h = np.abs(GY * W)
        term = rstd[:, None] * (h + h.mean(axis=1, keepdims=True)
                                + np.abs(xhat) * (h * np.abs(xhat)).mean(axis=1, keepdims=True))
        held(download(gx), GX, N * U * 4 * term + half_ulp(dt, GX), "grad_x")
        Nw = rows + 300
        # xhat itself carries the rounding of x - mean: |x| + |mean| in units of 1 / rstd
        carry = (np.abs(X) + np.abs(mean[:, None])) * rstd[:, None]
        held(download(gw), GW, U * ((Nw * np.abs(GY * xhat)).sum(0) + 4 * (np.abs(GY) * carry).sum(0))
             + half_ulp(dt, GW), "grad_weight")
        if bias:
            held(download(gb), GB, U * Nw * np.abs(GY).sum(0) + half_ulp(dt, GB), "grad_bias")
        else:
            assert gb is None
        again = ops.dora_layernorm_backward(gy, x, w, torch.from_numpy(mean32).cuda(),
                                            torch.from_numpy(rstd32).cuda(), need=need)
        for a, g in zip(again, (gx, gw, gb)):
            assert (a is None and g is None) or torch.equal(a, g)   # fixed order, same bits


def test_gradients_against_differences(ops):
    """d(sum gy y) / d(x, w, b) by central differences of the float64 forward."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 11)).astype(np.float32)
    w = (1 + 0.3 * rng.standard_normal(11)).astype(np.float32)
    b = rng.standard_normal(11).astype(np.float32)
    gy = rng.standard_normal((3, 11)).astype(np.float32)
    eps = 1e-3
    _, mean, rstd = ref.layernorm(x, w, b, eps)
    got = ops.dora_layernorm_backward(stored(gy, torch.float32), stored(x, torch.float32),
                                      stored(w, torch.float32), stored(mean, torch.float32),
                                      stored(rstd, torch.float32))
    args = [a.astype(np.float64) for a in (x, w, b)]
    for k, g in enumerate(got):
        diff = np.zeros_like(args[k])
        for i in np.ndindex(args[k].shape):
            vals = []
            for d in (1e-5, -1e-5):
                moved = [a.copy() for a in args]
                moved[k][i] += d
                vals.append(np.sum(gy * ref.layernorm(*moved, eps)[0]))
            diff[i] = (vals[0] - vals[1]) / 2e-5
        # float32 gradient terms of order 1 (1e-5), differences' own error (1e-8)
        assert np.max(np.abs(download(g) - diff)) <= 1e-5 * max(1.0, np.max(np.abs(diff)))


def test_constant_rows_nan_and_infinity_stay_in_their_rows(ops):
    x = torch.randn(6, 1000, device="cuda")
    x[1] = 3.0                       # variance 0: y = b
    x[2, 5] = float("nan")
    x[3, 999] = float("inf")
    w, b = torch.randn(1000, device="cuda"), torch.randn(1000, device="cuda")
    y, mean, rstd = ops.dora_layernorm(x, w, b, eps=1e-5)
    assert torch.equal(y[1], b) and mean[1] == 3.0
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    fine, _, _ = ops.dora_layernorm(x[[0, 4, 5]].contiguous(), w, b, eps=1e-5)
    assert torch.equal(y[[0, 4, 5]], fine)
    gy = torch.randn(6, 1000, device="cuda")
    gx, _, _ = ops.dora_layernorm_backward(gy, x, w, mean, rstd, need=("x",))
    assert torch.isnan(gx[2]).all() and torch.isfinite(gx[[0, 1, 4, 5]]).all()


def test_no_rows_no_weight_and_single_outputs(ops):
    x = torch.empty(0, 40, device="cuda")
    y, mean, rstd = ops.dora_layernorm(x)
    assert y.shape == (0, 40) and mean.shape == rstd.shape == (0,)
    gx, gw, gb = ops.dora_layernorm_backward(x, x, None, mean, rstd)
    assert gx.shape == (0, 40) and (gw == 0).all() and (gb == 0).all()
    x, gy = torch.randn(50, 300, device="cuda"), torch.randn(50, 300, device="cuda")
    ones = torch.ones(300, device="cuda")
    y, mean, rstd = ops.dora_layernorm(x)
    y1, _, _ = ops.dora_layernorm(x, ones, torch.zeros(300, device="cuda"))
    assert torch.equal(y, y1)
    full = ops.dora_layernorm_backward(gy, x, ones, mean, rstd)
    plain = ops.dora_layernorm_backward(gy, x, None, mean, rstd)
    for i, n in enumerate(("x", "weight", "bias")):
        assert torch.equal(full[i], plain[i])
        one = ops.dora_layernorm_backward(gy, x, None, mean, rstd, need=(n,))
        assert torch.equal(one[i], full[i])
        assert [k for k, t in enumerate(one) if t is not None] == [i]


def test_refusals(ops):
    x, w = torch.randn(4, 32, device="cuda"), torch.randn(32, device="cuda")
    with pytest.raises(ValueError, match="contiguous rows"):
        ops.dora_layernorm(x.t(), None)
    with pytest.raises(ValueError, match="overlap"):
        ops.dora_layernorm(x[0].expand(4, 32))
    with pytest.raises(ValueError, match="weight has shape"):
        ops.dora_layernorm(x, w[:31])
    with pytest.raises(ValueError, match="weight has dtype"):
        ops.dora_layernorm(x, w.bfloat16())
    with pytest.raises(ValueError, match="unsupported dtype"):
        ops.dora_layernorm(x.half())
    with pytest.raises(ValueError, match="device"):
        ops.dora_layernorm(x.cpu())
    with pytest.raises(ops.DoraError, match="DORA_ERR_FLAGS"):
        ops.dora_layernorm(x, w, eps=-1.0)
    y, mean, rstd = ops.dora_layernorm(x, w)
    with pytest.raises(ValueError, match="grad_y has shape"):
        ops.dora_layernorm_backward(x[:, :31], x, w, mean, rstd)
    with pytest.raises(ops.DoraError, match="DORA_ERR_WORKSPACE"):
        ops.dora_layernorm_backward(x, x, w, mean, rstd,
                                    workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_side_stream_and_graph(ops):
    x, gy = torch.randn(200, 1030, device="cuda").bfloat16(), torch.randn(200, 1030, device="cuda").bfloat16()
    w, b = torch.randn(1030, device="cuda").bfloat16(), torch.randn(1030, device="cuda").bfloat16()

    def step():
        y, mean, rstd = ops.dora_layernorm(x, w, b)
        return (y, mean, rstd, *ops.dora_layernorm_backward(gy, x, w, mean, rstd))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b_) for a, b_ in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        for t in out:
            t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b_) for a, b_ in zip(out, want))
        assert all(torch.equal(a, b_) for a, b_ in zip(step(), want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [1, 5, 70, 1001, 5121, 8200])
def test_gradient_of_constant_rows_whose_mean_times_rstd_overflows(ops, width, dtype):
    """Sums of 2^114 are exact, so xhat is 0 and the formula leaves the centred gradient; what a
    row's width leaves of the last threads must not bring in 0 - mean."""
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    x = torch.full((3, width), 2.0 ** 114, dtype=dt, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(width)
    gy = torch.randn(3, width, device="cuda", generator=gen).to(dt)
    _, mean, rstd = ops.dora_layernorm(x, None, None, eps=1e-12)
    assert torch.equal(mean, x[:, 0].float())
    gx, gw, gb = ops.dora_layernorm_backward(gy, x, None, mean, rstd)
    assert torch.count_nonzero(gw) == 0
    g = gy.double()
    want = rstd.double()[:, None] * (g - g.mean(1, keepdim=True))
    # float32 sums of terms below 6, then one rounding to the type (half a unit in the last place)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    assert ((gx.double() - want).abs() <= want.abs() * half + 2e-5 * rstd.double()[:, None]).all()
    assert ((gb.double() - g.sum(0)).abs() <= g.sum(0).abs() * half + 2e-6).all()


@pytest.mark.parametrize("rows,width", [(3, 8200), (300, 9001), (7, 10240), (5, 10241), (261, 12289),
                                        (2, 14336), (6, 14337), (300, 16383), (520, 16384), (4, 16385)])
def test_wide_bf16_rows(ops, rows, width):
    test_forward_and_backward(ops, rows, width, "bf16")


@pytest.mark.parametrize("width", [40, 200, 1031, 2300, 5121, 7168, 8192, 9001, 16384, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_alone_have_the_bits_they_have_together(ops, width, dtype):
    """Any subset of the three gradients, rows that do not fill a workgroup's last turn."""
    for rows in (1, 5, 2049):
        if rows * width > 1 << 25:
            continue
        say("layernorm", rows, width, dtype)
        x, gy, w, _ = make(rows, width, DT[dtype], rows + width, False, True)
        _, mean, rstd = ops.dora_layernorm(x, w, None)
        full = ops.dora_layernorm_backward(gy, x, w, mean, rstd)
        for need in (("x",), ("weight",), ("bias",), ("weight", "bias"), ("x", "bias")):
            got = ops.dora_layernorm_backward(gy, x, w, mean, rstd, need=need)
            for name, a, b in zip(("x", "weight", "bias"), got, full):
                assert a is None if name not in need else torch.equal(a, b), (rows, need, name)
