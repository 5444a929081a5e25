"""Token log probabilities, entropies, top alternatives and their gradient against float64.

Bars.  u = 2^-24.  A difference l = scale (z - max) carries 2 roundings, so exp(l) is off by
2 u |l| + 2 u relative and the row's sum of exponentials by that much on average plus its chain of
additions, at most vocab / 256 + 32 of them; a logarithm adds its own rounding:
  logp      u (vocab / 256 + 64 + 8 (max l - l_target + log vocab))
  entropy   u (vocab / 256 + 64) (1 + 2 log vocab)
  lse       as logp's, plus 2 u |lse|
  gradient  relative to p (|ga| + |gh| (|log p + H| + 1)) scale:  u (64 + 8 |l| + 8 |lse|) from the
            float32 lse and entropy it is given, plus half a last place of its type
Indices are equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import finetune as ref
from tests.gpu_util import download

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NEG = float("-inf")


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from parameter_efficient_fine_dora_amd import ops as _ops, _lib
    _lib.lib()
    return _ops


def say(*a):
    print(*a, flush=True)


def held(got, want, bar, what):
    with np.errstate(invalid="ignore"):
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        bad = ~same & ~(np.abs(got - want) <= bar)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4])


def check(ops, z, y, scale=1.0, top=0):
    """Forward and backward of logits z (GPU, maybe strided) against float64."""
    Z, Yt = download(z), y.cpu().numpy()
    T, V = Z.shape
    logp, H, lse, tl, ti = ref.token_logprob(Z, Yt, scale, top)
    got = ops.dora_token_logprob(z, y, scale=scale, top=top)
    live = (Yt >= 0) & (Yt < V)
    base = V / 256 + 64
    with np.errstate(invalid="ignore"):
        gap = np.where(live, scale * (Z.max(axis=1) - Z[np.arange(T), np.where(live, Yt, 0)]), 0.0)
    bar = U * (base + 8 * (np.where(np.isfinite(gap), gap, 0.0) + np.log(V)))
    held(download(got[0]), logp, bar, "logp")
    held(download(got[1]), H, U * base * (1 + 2 * np.log(V)), "entropy")
    held(download(got[2]), lse, bar + 2 * U * np.abs(np.where(np.isfinite(lse), lse, 0)), "lse")
    if top:
        assert np.array_equal(got[4].cpu().numpy(), ti), "top_index"
        with np.errstate(invalid="ignore"):
            low = np.where(np.isfinite(tl), np.abs(tl), 0.0)
        held(download(got[3]), tl, U * (base + 8 * (low + np.log(V))), "top_logp")
    else:
        assert got[3] is None and got[4] is None

    rng = np.random.default_rng(V + T)
    ga = rng.standard_normal(T).astype(np.float32)
    gh = rng.standard_normal(T).astype(np.float32)
    G = ref.token_logprob_backward(ga, gh, Z, Yt, scale)
    guard = torch.full((T * V + 16,), 7.0, dtype=z.dtype, device="cuda")
    g = ops.dora_token_logprob_backward(torch.from_numpy(ga).cuda(), torch.from_numpy(gh).cuda(), z,
                                        y, got[2], got[1], scale=scale,
                                        grad_logits=guard[8:8 + T * V].view(T, V))
    assert (guard[:8] == 7).all() and (guard[8 + T * V:] == 7).all()
    with np.errstate(invalid="ignore", over="ignore"):
        l = np.where(np.isfinite(Z), Z, 0.0) * scale
        lp = np.where(np.isfinite(Z), Z * scale - lse[:, None], -np.inf)
        p = np.exp(lp)
        Hc = np.where(np.isfinite(H), H, 0.0)[:, None]
        mag = p * (np.abs(ga[:, None]) + np.abs(gh[:, None])
                   * (np.where(np.isfinite(lp), np.abs(lp), 0.0) + np.abs(Hc) + 1)) * scale
        fin = np.where(np.isfinite(lse), np.abs(lse), 0.0)[:, None]
        # the entropy it is given is off by its own bar
        rel = U * (64 + 8 * np.abs(l) + 8 * fin + base * (1 + 2 * np.log(V)))
        rel = np.where(np.isfinite(rel), rel, 0.0)
        half = np.abs(G) * (2.0 ** -8 if z.dtype == torch.bfloat16 else U)
        bar = mag * rel + half + 2 * U * np.abs(ga[:, None]) * scale * (p > 0)
    held(download(g), G, bar, "grad_logits")
    return got, g


def logits(T, V, dt, seed, ld=None, std=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ld = ld or V
    buf = torch.full((T, ld), float("nan"), dtype=dt, device="cuda")
    buf[:, :V] = (torch.randn(T, V, device="cuda", generator=g) * std).to(dt)
    y = torch.randint(V, (T,), device="cuda", generator=g)
    return buf[:, :V], y


SIZES = [(1, 1, 1), (3, 2, 2), (2, 7, 8), (5, 64, 64), (1, 255, 255), (4, 257, 300), (33, 1000, 1000),
         (1, 4096, 4096), (7, 5003, 5008), (1, 32768, 32768), (2, 50021, 50048), (1, 131072, 131072),
         (3, 262147, 262147), (65, 8192, 8192), (300, 777, 777), (1100, 513, 520)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,ld", SIZES)
def test_sizes(ops, T, V, ld, dtype):
    for scale, top in ((1.0, 0), (1.25, min(V, 20))):
        say("logprob", T, V, ld, dtype, scale, top)
        z, y = logits(T, V, DT[dtype], T + V, ld)
        check(ops, z, y, scale, top)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [1, 2, 5, 31, 64])
def test_top_with_ties_in_index_order(ops, top, dtype):
    """Few distinct values, so every rank is a tie; descending and ascending rows."""
    for T, V in ((3, 64), (4, 3001), (2, 70000)):
        say("ties", T, V, top, dtype)
        g = torch.Generator(device="cuda")
        g.manual_seed(V)
        z = torch.randint(-2, 3, (T, V), device="cuda", generator=g).to(DT[dtype])
        z[0] = 0.0
        z[1] = torch.arange(V, device="cuda").to(DT[dtype])       # ascending, ties in bf16
        z[2 % T, ::2] *= -1.0                                      # -0 equals +0
        y = torch.randint(V, (T,), device="cuda", generator=g)
        got = ops.dora_token_logprob(z, y, top=top)
        want = ref.token_logprob(download(z), y.cpu().numpy(), 1.0, top)
        assert np.array_equal(got[4].cpu().numpy(), want[4])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_rows(ops, dtype):
    dt = DT[dtype]
    low = torch.finfo(dt).min
    for V in (40, 1001, 33000):
        say("masks", V, dtype)
        z, y = logits(9, V, dt, V)
        z[0] = NEG                                # nothing left
        z[1] = low                                # every logit the type's lowest: uniform
        z[2, 1:] = NEG                            # one left
        y[2] = 0
        z[3, V // 2:] = NEG                       # the target masked
        y[3] = V - 1
        z[4, V // 2:] = low
        y[4] = 1
        y[5] = -100                               # no target
        y[6] = V                                  # outside the vocabulary
        z[7, :] = NEG
        z[7, 5] = low                             # only a lowest value left
        y[7] = 5
        z[8] = z[8] * 100.0                       # |lse| in the hundreds or thousands
        k = min(V, 24)
        got, g = check(ops, z, y, 1.0, k)
        assert got[0][0] == NEG and got[1][0] == 0 and got[2][0] == NEG and (g[0] == 0).all()
        assert abs(float(got[0][1]) + np.log(V)) <= 1e-5 * np.log(V) + V * U
        assert got[0][2] == 0 and got[0][3] == NEG and got[0][7] == 0
        for t in (5, 6):
            assert got[0][t] == got[1][t] == got[2][t] == 0 and (got[4][t] == -1).all()
            assert (g[t] == 0).all()
        # the uniform row's gradient: ga (1[j = y] - 1 / V), the entropy's share vanishes
        ga = torch.ones(9, device="cuda")
        u = download(ops.dora_token_logprob_backward(ga, None, z, y, got[2], got[1]))[1]
        want = -np.full(V, 1.0 / V)
        want[int(y[1])] += 1.0
        assert np.max(np.abs(u - want)) <= 2.0 ** -8 * np.max(np.abs(want)) + 1e-6
        # a scale above 1 takes the lowest value past the type's range
        s = ops.dora_token_logprob(z, y, scale=1.5, top=2)
        assert abs(float(s[0][1]) + np.log(V)) <= 1e-5 * np.log(V) + V * U
        assert torch.isfinite(s[0][[2, 4, 8]]).all() and not torch.isnan(torch.stack(s[:3])).any()
        gs = ops.dora_token_logprob_backward(ga, ga, z, y, s[2], s[1], scale=1.5)
        assert torch.isfinite(gs.float()).all()


def test_nan_and_infinity_stay_in_their_rows(ops):
    for V in (50, 20001):
        z, y = logits(6, V, torch.float32, V)
        z[1, 7] = float("nan")
        z[2, V - 1] = float("inf")
        z[4] = NEG
        z[4, 3] = float("nan")
        got = ops.dora_token_logprob(z, y, top=3)
        for t in (1, 2, 4):
            assert all(torch.isnan(got[k][t]) for k in (0, 1, 2)), t
        assert got[4][1, 0] == 7 and got[4][2, 0] == V - 1 and got[4][4].tolist() == [3, 0, 1]
        keep = [0, 3, 5]
        fine = ops.dora_token_logprob(z[keep].contiguous(), y[keep].contiguous(), top=3)
        for a, b in zip(got, fine):
            assert torch.equal(a[keep], b)
        ga = torch.ones(6, device="cuda")
        g = ops.dora_token_logprob_backward(ga, ga, z, y, got[2], got[1])
        assert torch.isfinite(g[keep]).all() and torch.isnan(g[1]).any()


def test_gradient_against_differences(ops):
    rng = np.random.default_rng(3)
    z = (rng.standard_normal((3, 9)) * 2).astype(np.float32)
    z[1, 4] = -np.inf
    y = np.array([2, 0, 8])
    ga, gh = rng.standard_normal(3), rng.standard_normal(3)
    scale = 0.75
    zt, yt = torch.from_numpy(z).cuda(), torch.from_numpy(y).cuda()
    out = ops.dora_token_logprob(zt, yt, scale=scale)
    g = download(ops.dora_token_logprob_backward(torch.from_numpy(ga).float().cuda(),
                                                 torch.from_numpy(gh).float().cuda(), zt, yt, out[2],
                                                 out[1], scale=scale))
    for i in np.ndindex(z.shape):
        vals = []
        for d in (1e-5, -1e-5):
            m = z.astype(np.float64)
            m[i] += d
            lp, H = ref.token_logprob(m, y, scale)[:2]
            vals.append(np.sum(ga * lp + gh * H))
        assert abs(g[i] - (vals[0] - vals[1]) / 2e-5) <= 1e-5   # float32 terms of order 1


def test_optional_gradients_and_no_rows(ops):
    z, y = logits(5, 600, torch.float32, 8)
    out = ops.dora_token_logprob(z, y)
    ga, gh = torch.randn(5, device="cuda"), torch.randn(5, device="cuda")
    zero = torch.zeros(5, device="cuda")
    a = ops.dora_token_logprob_backward(ga, None, z, y, out[2], None)
    assert torch.equal(a, ops.dora_token_logprob_backward(ga, zero, z, y, out[2], out[1]))
    h = ops.dora_token_logprob_backward(None, gh, z, y, out[2], out[1])
    assert torch.equal(h, ops.dora_token_logprob_backward(zero, gh, z, y, out[2], out[1]))
    none = ops.dora_token_logprob_backward(None, None, z, y, out[2], None)
    assert (none == 0).all()
    e = ops.dora_token_logprob(z[:0], y[:0], top=4)
    assert e[0].shape == (0,) and e[4].shape == (0, 4)
    assert ops.dora_token_logprob_backward(ga[:0], None, z[:0], y[:0], out[2][:0], None).shape == (0, 600)


def test_refusals(ops):
    z, y = logits(4, 32, torch.float32, 1)
    with pytest.raises(ValueError, match="targets has dtype"):
        ops.dora_token_logprob(z, y.int())
    with pytest.raises(ValueError, match="targets has shape"):
        ops.dora_token_logprob(z, y[:3])
    with pytest.raises(ValueError, match="contiguous rows"):
        ops.dora_token_logprob(z.t(), y[:1].expand(32).contiguous())
    with pytest.raises(ValueError, match="unsupported dtype"):
        ops.dora_token_logprob(z.half(), y)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ops.DoraError, match="DORA_ERR_FLAGS"):
            ops.dora_token_logprob(z, y, scale=bad)
    for top in (33, 65):
        with pytest.raises(ops.DoraError, match="DORA_ERR_SHAPE"):
            ops.dora_token_logprob(z, y, top=top)
    out = ops.dora_token_logprob(z, y)
    with pytest.raises(ops.DoraError, match="DORA_ERR_NULL"):
        ops.dora_token_logprob_backward(None, out[0], z, y, out[2], None)
    with pytest.raises(ValueError, match="contiguous"):
        ops.dora_token_logprob_backward(out[0][:1].expand(4), None, z, y, out[2], None)


def test_side_stream_and_graph(ops):
    z, y = logits(70, 9001, torch.bfloat16, 4)
    ga = torch.randn(70, device="cuda")

    def step():
        out = ops.dora_token_logprob(z, y, scale=0.9, top=6)
        return (*out, ops.dora_token_logprob_backward(ga, ga, z, y, out[2], out[1], scale=0.9))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        for t in out:
            t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,top", [(3, 1500, 20), (5, 2048, 64), (2, 2049, 64), (3, 6000, 33),
                                     (2, 8192, 64), (40, 8193, 5), (1100, 4100, 7), (1050, 9000, 64)])
def test_top_of_every_arrangement(ops, T, V, top, dtype):
    """Rows of one wave, of one workgroup and cut into chunks, each held in registers or streamed:
    random rows, constant ones (every element a tie), one whose largest lie together at its end,
    and rows of few distinct values with most of them masked."""
    say("arrangements", T, V, top, dtype)
    z, y = logits(T, V, DT[dtype], 7 * V + T)
    z[0] = 1.5
    if T > 1:
        z[1] = torch.linspace(-4, 4, V, device="cuda").to(DT[dtype])
    if T > 2:
        z[2] = (torch.arange(V, device="cuda") % 3).to(DT[dtype])
        z[2, torch.arange(V, device="cuda") % 50 != 0] = NEG
    rows = sorted({0, min(1, T - 1), min(2, T - 1), T // 2, T - 1})
    got = ops.dora_token_logprob(z, y, top=top)
    want = ref.token_logprob(download(z[rows].contiguous()), y[rows].cpu().numpy(), 1.0, top)
    assert np.array_equal(got[4][rows].cpu().numpy(), want[4])
    base = V / 256 + 64
    low = np.where(np.isfinite(want[3]), np.abs(want[3]), 0.0)
    held(download(got[3][rows]), want[3], U * (base + 8 * (low + np.log(V))), "top_logp")
    held(download(got[1][rows]), want[1], U * base * (1 + 2 * np.log(V)), "entropy")


@pytest.mark.parametrize("T,V", [(1030, 50257), (6, 50257), (1100, 8193), (3, 16385), (1500, 3001)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_rows_bits_do_not_depend_on_its_address(ops, T, V, dtype):
    """Rows of an odd vocabulary start at every alignment; equal rows give equal bits, wherever
    the first of them starts."""
    say("addresses", T, V, dtype)
    one = (torch.randn(V, device="cuda") * 3).to(DT[dtype])
    y = torch.full((T,), 11, device="cuda")
    ga = torch.full((T,), 0.5, device="cuda")
    seen = []
    for start in (0, 1, 2):
        buf = torch.full((T * V + 8,), float("nan"), dtype=DT[dtype], device="cuda")
        z = buf[start:start + T * V].view(T, V)
        z[:] = one
        got = ops.dora_token_logprob(z, y, top=4)
        g = ops.dora_token_logprob_backward(ga, ga, z, y, got[2], got[1])
        for t in (*got, g):
            assert torch.equal(t, t[:1].expand_as(t))
        seen.append([t[0].clone() for t in (*got, g)])
    for later in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], later))
