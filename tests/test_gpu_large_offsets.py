"""Layer norm, token log probabilities and AdamW where element offsets pass 32 bits and where rows
outnumber a launch's grid.  The rows or elements on both sides of the mark are compared with the
same call on a small copy of them, bit for bit."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from parameter_efficient_fine_dora_amd import ops as _ops, _lib
    _lib.lib()
    return _ops


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def say(*a):
    print(*a, flush=True)


def test_logprob_past_32_bits(ops):
    T, V = 16500, 131072                      # 2.16e9 logits, 4.3 GB
    say("logprob", T, V)
    z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 7, 16383, 16384, T - 1], device="cuda")
    z[rows] = torch.randn(5, V, device="cuda").bfloat16()
    y = torch.full((T,), -100, device="cuda")
    y[rows] = torch.tensor([5, V - 1, 0, 9, 100], device="cuda")
    got = ops.dora_token_logprob(z, y, top=3)
    small = z[rows].contiguous()
    yy = y[rows].contiguous()
    one = [ops.dora_token_logprob(z[r:r + 1], y[r:r + 1], top=3) for r in rows.tolist()]
    for a, b in zip(got, ops.dora_token_logprob(small, yy, top=3)):
        assert torch.allclose(a[rows].double(), b.double(), rtol=1e-5, atol=1e-5)
    for k in range(5):                        # a row alone is split over workgroups
        assert torch.allclose(torch.cat([o[k] for o in one]).double(), got[k][rows].double(),
                              rtol=1e-5, atol=1e-5)
    skipped = torch.ones(T, dtype=torch.bool, device="cuda")
    skipped[rows] = False
    assert (got[0][skipped] == 0).all() and (got[4][skipped] == -1).all()
    ga = torch.randn(T, device="cuda")
    g = ops.dora_token_logprob_backward(ga, None, z, y, got[2], None)
    gs = ops.dora_token_logprob_backward(ga[rows].contiguous(), None, small, yy,
                                         got[2][rows].contiguous(), None)
    assert torch.equal(g[rows], gs)
    assert not g[skipped][::500].any()


def test_logprob_more_rows_than_a_grid_column(ops):
    T, V = 70001, 40
    say("logprob", T, V)
    z = torch.randn(T, V, device="cuda")
    y = torch.randint(V, (T,), device="cuda")
    got = ops.dora_token_logprob(z, y, top=2)
    ga = torch.randn(T, device="cuda")
    g = ops.dora_token_logprob_backward(ga, ga, z, y, got[2], got[1])
    cut = slice(65000, T)
    part = ops.dora_token_logprob(z[cut].contiguous(), y[cut].contiguous(), top=2)
    for a, b in zip(got, part):
        assert torch.equal(a[cut], b)
    assert torch.equal(g[cut], ops.dora_token_logprob_backward(
        ga[cut].contiguous(), ga[cut].contiguous(), z[cut].contiguous(), y[cut].contiguous(), part[2],
        part[1]))


def test_layernorm_past_32_bits_and_past_a_grid(ops):
    for R, D in ((263000, 8192), ((1 << 21) + 77, 24)):
        say("layernorm", R, D)
        x = torch.ones(R, D, dtype=torch.bfloat16, device="cuda")
        edge = [0, 1, R // 2, 262143, 262144, R - 2, R - 1]
        rows = torch.tensor(sorted(r for r in edge if r < R), device="cuda")
        x[rows] = torch.randn(len(rows), D, device="cuda").bfloat16()
        w, b = torch.randn(D, device="cuda").bfloat16(), torch.randn(D, device="cuda").bfloat16()
        y, mean, rstd = ops.dora_layernorm(x, w, b)
        small = x[rows].contiguous()
        ys, ms, rs = ops.dora_layernorm(small, w, b)
        assert torch.equal(y[rows], ys) and torch.equal(mean[rows], ms) and torch.equal(rstd[rows], rs)
        gx, gw, gb = ops.dora_layernorm_backward(y, x, w, mean, rstd)
        gxs, _, _ = ops.dora_layernorm_backward(ys, small, w, ms, rs)
        assert torch.equal(gx[rows], gxs)
        want = torch.zeros(D, dtype=torch.float64, device="cuda")
        for r0 in range(0, R, 1 << 17):       # the columns' sums of y, in float64
            want += y[r0:r0 + (1 << 17)].double().sum(0)
        assert torch.allclose(gb.double(), want, rtol=2 ** -7, atol=1e-3 * float(want.abs().max()))
        del x, y, gx, gw, gb


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_past_32_bits(ops, bits):
    n = (1 << 31) + 5000
    say("adamw", n, bits)
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    small = bits == 8
    m = torch.zeros(n, dtype=torch.int8 if small else torch.float32, device="cuda")
    v = torch.zeros(n, dtype=torch.uint8 if small else torch.float32, device="cuda")
    blocks = -(-n // 128)
    sc = [torch.zeros(blocks, device="cuda") for _ in range(2)] if small else [None, None]
    cut = slice((1 << 31) - 4096, n)           # starts at a block of 128
    k = cut.stop - cut.start
    p[cut] = torch.randn(k, device="cuda").bfloat16()
    g[cut] = torch.randn(k, device="cuda").bfloat16()
    bcut = slice(cut.start // 128, blocks)
    ref = [t[cut].clone() for t in (p, m, v)] + ([s[bcut].clone() for s in sc] if small else [])
    gr = g[cut].clone()

    def plan(p, m, v, s):
        return ops.AdamWPlan([p], [m], [v], **(dict(exp_avg_scales=[s[0]], exp_avg_sq_scales=[s[1]])
                                               if small else {}))

    norm = ops.dora_adamw(plan(p, m, v, sc), [g], step=1, lr=1e-2, max_norm=1.0)
    norm_s = ops.dora_adamw(plan(*ref[:3], ref[3:]), [gr], step=1, lr=1e-2, max_norm=1.0)
    assert abs(float(norm) - float(norm_s)) <= 1e-6 * float(norm_s)
    # the norm's sums are grouped differently, so the clipped gradient may differ in its last bit
    assert torch.allclose(p[cut].float(), ref[0].float(), rtol=2 ** -7, atol=1e-7)
    assert not p[:1 << 20].any()
    if small:
        a = ops.dora_adamw_dequantize(m, sc[0])[cut]
        b = ops.dora_adamw_dequantize(ref[1], ref[3])
        assert torch.allclose(a, b, rtol=0.05, atol=1e-6)
    else:
        assert torch.allclose(m[cut], ref[1], rtol=1e-5, atol=0)
