"""Preference and policy losses on the GPU against their float64 definitions: padded and packed
sequences, empty ones, masks that leave nothing, repeated and absent pairs.

Terms and sums are float64, so a result is off by its own rounding, 2^-24 of it, and by what float64
sums lose (2^-52 of the summands' magnitudes for each of at most a few thousand additions in a row,
under 1e-12 of them).  Gradients are formed from logits and weights as the forward returned them.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import posttrain as oracle

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24 * (1 + 1e-6)
PACKED = {
    "short": [3, 1, 7],
    "empty": [0, 0, 1, 0, 5, 300, 0, 0],
    "ones": [1] * 700,
    "rounds": [255, 1, 256, 257, 0, 1024, 3, 512],
    "long": [5000, 0, 1, 90001, 17],
}


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    from parameter_efficient_fine_dora_amd import _lib, ops
    _lib.lib()
    return ops


def near(got, want, scale=0.0, half=HALF):
    got = got.double().cpu().numpy().reshape(-1)
    want = np.asarray(want, np.float64).reshape(-1)
    assert got.shape == want.shape
    # a value below float32's normal range keeps an absolute half step
    bad = ~(np.abs(got - want) <= half * np.abs(want) + 1e-12 * scale + 2.0 ** -149)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


def dev(a, shape=None, odd=False):
    """On the GPU; `odd`: one element behind an allocation's start."""
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a))
    if odd:
        room = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        room[1:] = t.reshape(-1).cuda()
        t = room[1:]
    return t.cuda().view(shape or a.shape)


def batch(layout, seed, mask="some", lead=0, behind=0):
    """(logp, other maker, mask, offsets, spans, shape) of a layout: (S, L) or lengths."""
    rng = np.random.default_rng(seed)
    if isinstance(layout, tuple):
        shape, offsets = layout, None
    else:
        offsets = lead + np.concatenate([[0], np.cumsum(layout)]).astype(np.int64)
        shape = (int(offsets[-1]) + behind,)
    n = int(np.prod(shape))
    where = oracle.spans(shape, offsets)
    live = None
    if mask != "none":
        live = rng.random(n) < 0.7
        if mask == "rows":              # every other sequence has nothing left
            for a, b in where[::2]:
                live[a:b] = False
        if mask == "nothing":
            live[:] = False
    logp = (-3.0 * rng.random(n) ** 2 - 1e-3).astype(np.float32)

    def other(step):
        return (logp + step * rng.standard_normal(n)).astype(np.float32)

    return rng, n, logp, other, live, offsets, where, shape


def spoil(a, live):
    """NaN and infinities where a token does not count."""
    if a is None or live is None:
        return a
    a = a.copy()
    a[~live] = np.resize(np.array([np.nan, np.inf, -np.inf], np.float32), int((~live).sum()))
    return a


def check_preference(ops, layout, seed=0, mask="some", ref=True, kind="sigmoid", normalize=False,
                     lead=0, behind=0, odd=False, pairs=None, **how):
    rng, n, logp, other, live, offsets, where, shape = batch(layout, seed, mask, lead, behind)
    S = len(where)
    refp = other(0.3) if ref else None
    if pairs is None:
        pairs = rng.integers(0, S, (2, 2 * S + 1))
    chosen, rejected = (np.asarray(p, np.int64) for p in pairs)
    how = dict(kind=kind, normalize=normalize, **how)
    d_mask = None if live is None else dev(live, shape, odd)
    d_off = None if offsets is None else dev(offsets)
    c, r = dev(chosen), dev(rejected)
    got = ops.dora_preference_loss(dev(spoil(logp, live), shape, odd), c, r, mask=d_mask,
                                   ref_logp=dev(spoil(refp, live), shape, odd) if ref else None,
                                   offsets=d_off, **how)
    want = oracle.preference_loss(logp, chosen, rejected, where, refp, live, **how)
    beta = how.get("beta", 0.1)
    scale = beta * np.abs(logp.astype(np.float64) - (refp if ref else 0)).sum() + 1
    near(got[1], want[1], scale)
    near(got[2], want[2], scale)
    near(got[3], want[3])
    # the value's slope times the logit's error
    steep = 2 * (np.abs(want[2]).max(initial=1.0) + 1) / beta ** 2 if kind == "square" else 1.0
    near(got[0], want[0], scale * steep)
    gl = rng.standard_normal(len(chosen)).astype(np.float32)
    grad = ops.dora_preference_loss_backward(dev(gl), got[2], got[3], c, r, shape=shape, mask=d_mask,
                                             offsets=d_off, **how)
    how.pop("margin", None)
    wg = oracle.preference_backward(gl, got[2].cpu().numpy(), want[3], chosen, rejected, where, n, live,
                                    **how)
    # a sequence's pairs may cancel: their float64 sum loses 1e-12 of its terms at most
    near(grad, wg, np.abs(gl).sum() * beta * steep * (np.abs(want[2]).max(initial=0) + 1))
    assert grad.shape == torch.Size(shape)


@pytest.mark.parametrize("layout", [(1, 1), (2, 512), (3, 257), (5, 1), (61, 103), (2, 40001),
                                    *PACKED.values()], ids=str)
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "square"])
def test_preference(ops, layout, kind):
    if isinstance(layout, list) and len(layout) > 100:
        pairs = np.random.default_rng(3).integers(0, len(layout), (2, 50))
    else:
        pairs = None
    check_preference(ops, layout, 1, kind=kind, normalize=kind != "sigmoid", ref=kind != "hinge",
                     pairs=pairs)


@pytest.mark.parametrize("mask", ["none", "rows", "nothing"])
@pytest.mark.parametrize("normalize", [False, True])
def test_preference_masks(ops, mask, normalize):
    for layout in ((7, 300), PACKED["empty"], PACKED["rounds"]):
        check_preference(ops, layout, 2, mask=mask, normalize=normalize, smoothing=0.1)


def test_preference_options_and_alignment(ops):
    for odd in (False, True):
        for how in (dict(margin=0.7), dict(margin=-2.0, smoothing=1.0), dict(beta=3.0, smoothing=0.5),
                    dict(beta=1e-3, kind="square"), dict(beta=2.5, kind="hinge", margin=0.25)):
            check_preference(ops, PACKED["rounds"], 4, odd=odd, lead=3, behind=301, **how)


def test_preference_pairs_that_repeat_or_are_absent(ops):
    S = 6
    pairs = [[0, 0, 0, 5, 2, -1, 3, 6, 2 ** 40, 4], [1, 1, 2, 5, 0, 1, S, 2, 0, -2 ** 40]]
    check_preference(ops, (S, 77), 5, pairs=pairs)
    check_preference(ops, (S, 77), 5, pairs=[[], []])
    # more pairs than one look of a workgroup, and more sequences than one workgroup has threads
    rng = np.random.default_rng(6)
    check_preference(ops, (300, 9), 6, pairs=rng.integers(0, 300, (2, 1111)))


def test_no_sequences_and_no_tokens(ops):
    none = torch.empty(0, 5, device="cuda")
    e = torch.empty(0, dtype=torch.int64, device="cuda")
    one = torch.zeros(1, dtype=torch.int64, device="cuda")
    loss, score, logit, count = ops.dora_preference_loss(none, one, one)
    assert loss.tolist() == [0.0] and score.numel() == count.numel() == 0
    loss, score, _, count = ops.dora_preference_loss(torch.empty(3, 0, device="cuda"), one, one + 1)
    assert score.tolist() == count.tolist() == [0.0] * 3 and abs(float(loss[0]) - math.log(2)) < 1e-6
    packed = torch.ones(40, device="cuda")
    off = torch.tensor([7], device="cuda")          # no sequences among forty tokens
    loss, score, logit, count = ops.dora_preference_loss(packed, one, one, offsets=off)
    assert loss.tolist() == [0.0]
    g = ops.dora_preference_loss_backward(loss + 1, logit, count, one, one, shape=(40,), offsets=off)
    assert not g.any()
    value, stats, weight = ops.dora_policy_loss(packed, packed, packed, offsets=off, reduce="sequence")
    assert float(value) == 0.0 and not stats.any() and weight.numel() == 0
    g = ops.dora_policy_loss_backward(value + 1, weight, packed, packed, packed, offsets=off,
                                      reduce="sequence")
    assert not g.any()
    value, stats, weight = ops.dora_policy_loss(none, none, torch.empty(0, device="cuda"))
    assert float(value) == 0.0 and weight.tolist() == [1.0]
    assert ops.dora_policy_loss_backward(value, weight, none, none, none).shape == (0, 5)
    assert ops.dora_preference_loss(none, e, e)[0].numel() == 0


def check_policy(ops, layout, seed=0, mask="some", ref=True, per=False, reduce="token", lead=0,
                 behind=0, odd=False, spread=0.4, denominator=None, **how):
    rng, n, logp, other, live, offsets, where, shape = batch(layout, seed, mask, lead, behind)
    old, refp = other(spread), other(0.5) if ref else None
    adv = rng.standard_normal(len(where) if per else n).astype(np.float32)
    adv[rng.random(adv.size) < 0.1] = 0.0
    kw = dict(how, reduce=reduce, denominator=denominator, kl_coef=0.3 if ref else 0.0)
    okw = dict(kw)
    okw["dual"] = okw.pop("dual_clip", None) or math.inf
    value, ostats, oweight, ograd = oracle.policy_loss(logp, old, adv, where, refp, live, **okw)
    d = dict(mask=None if live is None else dev(live, shape, odd),
             offsets=None if offsets is None else dev(offsets),
             ref_logp=dev(spoil(refp, live), shape, odd) if ref else None, **kw)
    args = [dev(spoil(logp, live), shape, odd), dev(spoil(old, live), shape, odd),
            dev(adv, None, odd) if per else dev(spoil(adv, live), shape, odd)]
    loss, stats, weight = ops.dora_policy_loss(*args, **d)
    # summands are at most |A| rho + kl_coef kl
    scale = (np.abs(adv).max(initial=0) * math.exp(6 * spread) + 10) * max(1.0, n * oweight.max(initial=0))
    near(loss, value, scale)
    near(stats, ostats, 10 + math.exp(6 * spread))
    near(weight, oweight)
    grad = ops.dora_policy_loss_backward(torch.full((), -0.7, device="cuda"), weight, *args, **d)
    # the weight's rounding and the result's
    near(grad, np.float32(-0.7).astype(np.float64) * ograd, half=2 * HALF)
    assert grad.shape == torch.Size(shape)


@pytest.mark.parametrize("layout", [(1, 1), (8, 256), (3, 257), (61, 103), (2, 9001),
                                    *PACKED.values()], ids=str)
@pytest.mark.parametrize("reduce", ["token", "sequence"])
@pytest.mark.parametrize("per", [False, True], ids=["each", "per-sequence"])
def test_policy(ops, layout, reduce, per):
    check_policy(ops, layout, 1, reduce=reduce, per=per, ref=per)


@pytest.mark.parametrize("mask", ["none", "rows", "nothing"])
@pytest.mark.parametrize("reduce", ["token", "sequence"])
def test_policy_masks(ops, mask, reduce):
    for layout in ((7, 300), PACKED["empty"], PACKED["rounds"]):
        check_policy(ops, layout, 2, mask=mask, reduce=reduce, per=True)


@pytest.mark.parametrize("how", [dict(clip=(0.0, 0.0)), dict(clip=(1.0, math.inf)),
                                 dict(clip=(0.1, 0.3), dual_clip=1.5), dict(dual_clip=1.0),
                                 dict(denominator=1234.5)], ids=str)
def test_policy_bounds_and_alignment(ops, how):
    for odd in (False, True):
        for reduce in ("token", "sequence"):
            check_policy(ops, PACKED["rounds"], 3, odd=odd, lead=3, behind=301, reduce=reduce, **how)


def test_policy_counts_the_reference_without_a_coefficient(ops):
    logp, ref = -torch.rand(4, 50, device="cuda"), -torch.rand(4, 50, device="cuda")
    adv = torch.randn(4, device="cuda")
    a = ops.dora_policy_loss(logp, logp, adv, ref_logp=ref)
    b = ops.dora_policy_loss(logp, logp, adv)
    d = (ref - logp).double()
    assert torch.equal(a[0], b[0]) and float(b[1][0]) == 0.0
    near(a[1][0], float((torch.expm1(ref.double() - logp.double()) - (ref.double() - logp.double())).mean()), 1.0)


def test_policy_at_a_bound_and_far_from_it(ops):
    """Ratios of exactly the bound keep their slope; infinite ones are held, or give infinities; an
    advantage of 0 gives 0."""
    logp = torch.tensor([[0.0, 0.0, 800.0, 800.0, 800.0, 800.0]], device="cuda")
    old = torch.zeros(1, 6, device="cuda")
    adv = torch.tensor([[1.0, -1.0, 2.0, 0.0, -1.0, -3.0]], device="cuda")
    loss, stats, w = ops.dora_policy_loss(logp, old, adv, clip=(0.0, 0.0), reduce="token")
    g = ops.dora_policy_loss_backward(torch.ones((), device="cuda"), w, logp, old, adv, clip=(0.0, 0.0))
    assert g[0, :4].tolist() == [float(-w), float(w), 0.0, 0.0] and bool(torch.isinf(g[0, 4:]).all())
    assert float(loss) == math.inf
    loss, stats, w = ops.dora_policy_loss(logp, old, adv, clip=(0.0, 0.0), dual_clip=4.0)
    near(loss, (-1.0 + 1.0 - 2.0 + 0.0 + 4.0 + 12.0) / 6)
    g = ops.dora_policy_loss_backward(torch.ones((), device="cuda"), w, logp, old, adv, clip=(0.0, 0.0),
                                      dual_clip=4.0)
    assert g[0, 2:].tolist() == [0.0] * 4


def test_infinities_and_nan_of_counted_tokens(ops):
    """A counted token's infinity or NaN reaches its own sequence and pairs only."""
    logp = -torch.rand(6, 40, device="cuda")
    logp[0, 3], logp[2, 5] = -math.inf, math.nan
    c, r = (torch.tensor(v, device="cuda") for v in ([0, 1, 2, 4], [1, 0, 3, 5]))
    loss, score, logit, count = ops.dora_preference_loss(logp, c, r)
    assert score[0] == -math.inf and score[2].isnan() and torch.isfinite(score[[1, 3, 4, 5]]).all()
    assert loss[0] == math.inf and loss[1] == 0.0 and loss[2].isnan() and torch.isfinite(loss[3])
    g = ops.dora_preference_loss_backward(torch.ones(4, device="cuda"), logit, count, c, r, shape=(6, 40))
    near(g[0], np.full(40, -0.1)), near(g[1], np.full(40, 0.1))
    assert g[2:4].isnan().all() and torch.isfinite(g[4:]).all()


def test_more_tokens_than_one_round_a_wave(ops):
    """Chunks of several rounds: 1.3 million tokens, sequences of every length among them."""
    rng = np.random.default_rng(7)
    lengths = [0, 700001, 1, 0, *rng.integers(1, 3000, 300).tolist(), 255, 100003]
    off = torch.tensor(np.concatenate([[5], 5 + np.cumsum(lengths)]), device="cuda")
    n = int(off[-1]) + 999
    g = torch.Generator(device="cuda").manual_seed(1)
    logp = -torch.rand(n, device="cuda", generator=g)
    old = logp + 0.2 * torch.randn(n, device="cuda", generator=g)
    mask = torch.rand(n, device="cuda", generator=g) < 0.8
    S = len(lengths)
    c, r = torch.arange(S, device="cuda"), torch.arange(S, device="cuda").flip(0).contiguous()
    loss, score, logit, count = ops.dora_preference_loss(logp, c, r, ref_logp=old, mask=mask, offsets=off)
    d = torch.where(mask, logp.double() - old.double(), 0.0)
    adv = torch.randn(S, device="cuda", generator=g)
    value, stats, weight = ops.dora_policy_loss(logp, old, adv, mask=mask, offsets=off, reduce="sequence")
    gl = torch.ones((), device="cuda")
    grad = ops.dora_policy_loss_backward(gl, weight, logp, old, adv, mask=mask, offsets=off,
                                         reduce="sequence")
    pg = ops.dora_preference_loss_backward(loss, logit, count, c, r, shape=(n,), mask=mask, offsets=off)
    at, total, live = off.tolist(), 0.0, 0
    for s in range(S):
        a, b = at[s], at[s + 1]
        near(score[s], 0.1 * float(d[a:b].sum()), float(0.1 * d[a:b].abs().sum()))
        m = mask[a:b]
        k = int(m.sum())
        assert float(count[s]) == k
        if k:
            ratio = torch.exp(logp[a:b].double() - old[a:b].double())
            A = float(adv[s])
            bounded = ratio.clamp(max=1.2) if A >= 0 else ratio.clamp(min=0.8)
            slope = torch.where(m & (bounded == ratio), -A * ratio, 0.0)
            total, live = total - A * float(bounded[m].mean()), live + 1
            near(grad[a:b], (slope * float(weight[s])).cpu().numpy(), half=HALF)
        assert bool((pg[a:b][~m] == 0).all()) and (not k or len(pg[a:b][m].unique()) == 1)
    near(value, total / live, 10.0)
    assert not grad[:5].any() and not grad[at[-1]:].any() and not pg[:5].any() and not pg[at[-1]:].any()


@pytest.mark.parametrize("layout", [[16384], [16385], [4096], [4097], [512] * 8, [128] * 32, [1] * 33 + [7],
                                    [1000] * 16, [700] * 21, [0] * 20 + [4000, 96]], ids=lambda v: f"{len(v)}x{max(v)}")
def test_batches_of_one_workgroup_and_just_more(ops, layout):
    """The same sums whichever way they are formed: sequences on both sides of a batch that is not small."""
    g = torch.Generator(device="cuda").manual_seed(3)
    off = torch.tensor(np.concatenate([[0], np.cumsum(layout)]), device="cuda")
    n, S, more = int(off[-1]), len(layout), 20000
    logp, old, ref = (-torch.rand(n + more, device="cuda", generator=g) for _ in range(3))
    mask = torch.rand(n + more, device="cuda", generator=g) < 0.9
    adv = torch.randn(S + 1, device="cuda", generator=g)
    c, r = (torch.randint(0, S, (9,), device="cuda", generator=g) for _ in range(2))
    big = torch.cat([off, off[-1:] + more])
    a = ops.dora_preference_loss(logp[:n], c, r, ref_logp=ref[:n], mask=mask[:n], offsets=off)
    b = ops.dora_preference_loss(logp, c, r, ref_logp=ref, mask=mask, offsets=big)
    for x, y in zip(a, b):
        near(x, y[:x.numel()].double().cpu().numpy(), 10.0, half=2 * HALF)
    how = dict(kl_coef=0.1, reduce="sequence")
    v, stats, w = ops.dora_policy_loss(logp[:n], old[:n], adv[:S], ref_logp=ref[:n], mask=mask[:n], offsets=off, **how)
    v2, stats2, w2 = ops.dora_policy_loss(logp, old, adv, ref_logp=ref, mask=mask, offsets=big, **how)
    some = int((w > 0).sum())
    near(w * some, (w2[:S] * int((w2 > 0).sum())).double().cpu().numpy(), half=6 * HALF)
    # token sums are additive: of the batch, of what lies behind it, and of both
    one = dict(mask=mask[n:], offsets=torch.tensor([0, more], device="cuda"), denominator=1.0, kl_coef=0.1)
    rest = ops.dora_policy_loss(logp[n:], old[n:], adv[S:], ref_logp=ref[n:], **one)
    one = dict(denominator=1.0, kl_coef=0.1)
    part = ops.dora_policy_loss(logp[:n], old[:n], adv[:S], ref_logp=ref[:n], mask=mask[:n], offsets=off, **one)
    both = ops.dora_policy_loss(logp, old, adv, ref_logp=ref, mask=mask, offsets=big, **one)
    # three sums, each rounded to float32
    room = HALF * sum(abs(float(x[0])) for x in (part, rest, both)) + 1e-12 * (n + more)
    assert abs(float(part[0]) + float(rest[0]) - float(both[0])) <= room
    assert float(part[1][3]) + float(rest[1][3]) == float(both[1][3]) == int(mask.sum())
    means = [(float(x[1][0]) * float(x[1][3])) for x in (part, rest, both)]
    assert abs(means[0] + means[1] - means[2]) <= 6 * HALF * abs(means[2])


def test_more_than_2_32_tokens(ops):
    """Token numbers pass 2^32; the sequences' log ratios are 1/4 a token, and every fourth is masked."""
    n = 2 ** 32 + 5003
    at = [3, 2 ** 31 + 9, 2 ** 32 - 1, 2 ** 32 + 1, 2 ** 32 + 4999]
    off = torch.tensor(at, device="cuda")
    logp = torch.full((n,), -0.5, device="cuda")
    old = torch.full((n,), -0.75, device="cuda")
    mask = torch.ones(n, dtype=torch.bool, device="cuda")
    mask[::4] = False
    live = [b - a - ((b + 3) // 4 - (a + 3) // 4) for a, b in zip(at, at[1:])]
    c, r = torch.tensor([0, 2], device="cuda"), torch.tensor([1, 3], device="cuda")
    loss, score, logit, count = ops.dora_preference_loss(logp, c, r, ref_logp=old, mask=mask, offsets=off,
                                                         beta=1e-9)
    near(score, [0.25e-9 * v for v in live])
    near(count, live)
    gl = torch.ones(2, device="cuda")
    g = ops.dora_preference_loss_backward(gl, logit, count, c, r, shape=(n,), mask=mask, offsets=off, beta=1e-9)
    slope = [1e-9 / (1 + math.exp(float(h))) for h in logit]

    def ends(g, values):
        """The first and last counted tokens of each sequence, and those around them."""
        for s, v in enumerate(values):
            for t in {*range(at[s], at[s] + 5), *range(at[s + 1] - 5, at[s + 1])}:
                if at[s] <= t < at[s + 1]:
                    near(g[t], v if t % 4 else 0.0)
        assert not g[:at[0]].any() and not g[at[-1]:].any()
        # what a sequence holds beside its value and zero would change these
        total = sum(float(p.double().sum()) for p in g.split(2 ** 30))
        each = [v * k for v, k in zip(values, live)]
        assert abs(total - sum(each)) <= 1e-6 * sum(abs(v) for v in each)

    ends(g, [-slope[0], slope[0], -slope[1], slope[1]])
    del g
    adv = torch.tensor([1.0, -1.0, 0.5, 2.0], device="cuda")
    rho = math.exp(0.25)
    gain = [1.2, -rho, 0.6, 2.4]   # of 1 + 0.2, and the ratio itself for the negative advantage
    one = torch.ones((), device="cuda")
    for reduce in ("token", "sequence"):
        value, stats, w = ops.dora_policy_loss(logp, old, adv, mask=mask, offsets=off, reduce=reduce)
        by = [1 / sum(live)] * 4 if reduce == "token" else [0.25 / k for k in live]
        near(value, -sum(a * k * f for a, k, f in zip(gain, live, by)), 10.0)
        g = ops.dora_policy_loss_backward(one, w, logp, old, adv, mask=mask, offsets=off, reduce=reduce)
        w = w.expand(4).tolist()
        ends(g, [0.0, rho * w[1], 0.0, 0.0])


def test_offsets_that_are_wrong_touch_nothing_else(ops):
    """Decreasing, negative and too large offsets: any numbers, but none outside the tensors."""
    room = torch.full((3000,), 7.0, device="cuda")
    grad = room[1000:2000]
    logp = -torch.rand(1000, device="cuda")
    for off in ([500, 100, 900, 20], [-5, 10 ** 12, 3, 2000], [1000, 0, 1000, 0], [0, 0, 0, 0]):
        o = torch.tensor(off, device="cuda")
        c = torch.tensor([0, 1, 2], device="cuda")
        loss, score, logit, count = ops.dora_preference_loss(logp, c, c.flip(0).contiguous(), offsets=o)
        ops.dora_preference_loss_backward(loss, logit, count, c, c.flip(0).contiguous(), shape=(1000,),
                                          offsets=o, grad_logp=grad)
        adv = torch.ones(3, device="cuda")
        value, _, w = ops.dora_policy_loss(logp, logp, adv, offsets=o, reduce="sequence")
        ops.dora_policy_loss_backward(value, w, logp, logp, adv, offsets=o, reduce="sequence",
                                      grad_logp=grad)
        torch.cuda.synchronize()
        assert bool((room[:1000] == 7).all()) and bool((room[2000:] == 7).all())


def test_gradients_agree_with_differences(ops):
    """Central differences in float64 of the definition: steps of 1e-5 leave about 1e-9."""
    rng, n, logp, other, live, offsets, where, shape = batch([5, 0, 9, 4], 8)
    chosen, rejected = np.array([0, 2, 2]), np.array([2, 3, 0])
    old, ref, adv = other(0.3), other(0.3), rng.standard_normal(n).astype(np.float32)
    for kind in ("sigmoid", "square"):
        how = dict(kind=kind, beta=0.4, normalize=True)
        out = ops.dora_preference_loss(dev(logp), dev(chosen), dev(rejected), mask=dev(live),
                                       offsets=dev(offsets), margin=0.3, **how)
        gl = np.array([0.5, -1.0, 2.0], np.float32)
        got = ops.dora_preference_loss_backward(dev(gl), out[2], out[3], dev(chosen), dev(rejected),
                                                shape=shape, mask=dev(live), offsets=dev(offsets),
                                                margin=0.3, **how).cpu().numpy()

        def value(v):
            return float(oracle.preference_loss(v, chosen, rejected, where, None, live, margin=0.3,
                                                **how)[0] @ gl)
        _differences(value, logp, got)
    kw = dict(clip=(0.2, 0.28), kl_coef=0.3, reduce="sequence")
    args = dev(logp), dev(old), dev(adv)
    d = dict(ref_logp=dev(ref), mask=dev(live), offsets=dev(offsets), dual_clip=2.0, **kw)
    loss, _, w = ops.dora_policy_loss(*args, **d)
    got = ops.dora_policy_loss_backward(torch.ones((), device="cuda"), w, *args, **d).cpu().numpy()
    _differences(lambda v: oracle.policy_loss(v, old, adv, where, ref, live, dual=2.0, **kw)[0], logp, got)


def _differences(value, x, grad, step=1e-5):
    x = x.astype(np.float64)
    for t in range(x.size):
        up, down = x.copy(), x.copy()
        up[t] += step
        down[t] -= step
        d = (value(up) - value(down)) / (2 * step)
        assert abs(d - grad[t]) <= 1e-6 * max(1.0, abs(d)), (t, d, grad[t])


def test_same_bits_again_on_another_stream_and_from_a_graph(ops):
    rng, n, logp, other, live, offsets, where, shape = batch(PACKED["rounds"], 9)
    S = len(where)
    lp, old, ref, m, off = dev(logp), dev(other(0.3)), dev(other(0.2)), dev(live), dev(offsets)
    adv = torch.randn(S, device="cuda")
    c, r = dev(rng.integers(0, S, 9)), dev(rng.integers(0, S, 9))
    gl, one = torch.randn(9, device="cuda"), torch.ones((), device="cuda")

    def both():
        a = ops.dora_preference_loss(lp, c, r, ref_logp=ref, mask=m, offsets=off)
        g = ops.dora_preference_loss_backward(gl, a[2], a[3], c, r, shape=shape, mask=m, offsets=off)
        kw = dict(ref_logp=ref, mask=m, offsets=off, kl_coef=0.1, reduce="sequence")
        b = ops.dora_policy_loss(lp, old, adv, **kw)
        h = ops.dora_policy_loss_backward(one, b[2], lp, old, adv, **kw)
        return [*a, g, *b, h]

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for k in range(4):
        lp.mul_(1.01)
        want = both()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(held, want)), k


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_another_device_than_the_current_one(ops):
    def run(device):
        logp = torch.linspace(-3, -1, 80, device=device).view(4, 20)
        adv = torch.linspace(-1, 1, 4, device=device)
        c, r = torch.tensor([0, 2], device=device), torch.tensor([1, 3], device=device)
        a = ops.dora_preference_loss(logp, c, r)
        b = ops.dora_policy_loss(logp, logp - 0.1, adv)
        one = torch.ones((), device=device)
        return [*a, *b, ops.dora_preference_loss_backward(a[0], a[2], a[3], c, r, shape=(4, 20)),
                ops.dora_policy_loss_backward(one, b[2], logp, logp - 0.1, adv)]

    assert all(torch.equal(x.cpu(), y.cpu()) for x, y in zip(run("cuda:0"), run("cuda:1")))


def test_through_autograd(ops):
    """The functions with torch's own graph around them, against float64 on the CPU."""
    from parameter_efficient_fine_dora_amd.module import policy_loss, preference_loss, token_logprob
    torch.manual_seed(3)
    z = torch.randn(6, 20, 50, device="cuda", requires_grad=True)
    y = torch.randint(50, (6, 20), device="cuda")
    y[:, :5] = -100
    ref = -3 - torch.rand(6, 20, device="cuda")
    c, r = torch.tensor([0, 1, 2], device="cuda"), torch.tensor([3, 4, 5], device="cuda")
    logp = token_logprob(z, y)[0]
    loss, score = preference_loss(logp, c, r, ref_logp=ref, mask=y >= 0, normalize=True, beta=2.0)
    total, stats = policy_loss(logp.t().contiguous().t(), ref, torch.arange(6, device="cuda") - 2.5,
                               ref_logp=ref, mask=y >= 0, kl_coef=0.2, reduce="sequence")
    (loss.mean() + total).backward()
    zc = z.detach().double().cpu().requires_grad_()
    lp = zc.log_softmax(-1).gather(-1, y.clamp(min=0).cpu()[..., None])[..., 0]
    live, rc = (y >= 0).cpu(), ref.double().cpu()
    s = 2.0 * torch.where(live, lp - rc, 0).sum(1) / live.sum(1)
    ratio, adv = torch.exp(lp - rc), (torch.arange(6) - 2.5)[:, None]
    gain = torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv)
    l = -gain + 0.2 * (torch.expm1(rc - lp) - (rc - lp))
    want = -torch.nn.functional.logsigmoid(s[:3] - s[3:]).mean()
    want = want + (torch.where(live, l, 0).sum(1) / live.sum(1)).mean()
    want.backward()
    # chains through a softmax of 50 in float32
    assert float((z.grad.double().cpu() - zc.grad).abs().max()) <= 1e-5 * float(zc.grad.abs().max())
    assert abs(float(loss.mean() + total) - float(want)) <= 1e-5
    assert not score.requires_grad and not stats.requires_grad and float(stats[3]) == 90.0
    for bad in (dict(ref_logp=ref.clone().requires_grad_()),):
        with pytest.raises(ValueError, match="constant"):
            preference_loss(logp, c, r, **bad)
    with pytest.raises(ValueError, match="constant"):
        policy_loss(logp, ref, (torch.arange(6.0, device="cuda")).requires_grad_())


@pytest.mark.parametrize("call,message", [
    (lambda o, l, i: o.dora_preference_loss(l.double(), i, i), "dtype"),
    (lambda o, l, i: o.dora_preference_loss(l[:, ::2], i, i), "contiguous"),
    (lambda o, l, i: o.dora_preference_loss(l[0], i, i), "two dimensions"),
    (lambda o, l, i: o.dora_preference_loss(l, i, i, offsets=i), "one dimension"),
    (lambda o, l, i: o.dora_preference_loss(l[0], i, i, offsets=i.int()), "dtype"),
    (lambda o, l, i: o.dora_preference_loss(l, i, i[:1]), "shape"),
    (lambda o, l, i: o.dora_preference_loss(l, i.int(), i), "dtype"),
    (lambda o, l, i: o.dora_preference_loss(l, i, i, mask=l), "dtype"),
    (lambda o, l, i: o.dora_preference_loss(l, i, i, ref_logp=l[:2]), "shape"),
    (lambda o, l, i: o.dora_preference_loss(l, i, i, kind="other"), "expected one of"),
    (lambda o, l, i: o.dora_preference_loss(l, i, i, beta=0.0), "DORA_ERR_FLAGS"),
    (lambda o, l, i: o.dora_preference_loss(l, i, i, smoothing=1.5), "DORA_ERR_FLAGS"),
    (lambda o, l, i: o.dora_preference_loss(l, i, i, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
     "DORA_ERR_WORKSPACE"),
    (lambda o, l, i: o.dora_policy_loss(l, l[:2], l), "shape"),
    (lambda o, l, i: o.dora_policy_loss(l, l, l[0]), "shape"),
    (lambda o, l, i: o.dora_policy_loss(l, l, l, kl_coef=0.1), "needs ref_logp"),
    (lambda o, l, i: o.dora_policy_loss(l, l, l, clip=(1.5, 0.2)), "DORA_ERR_FLAGS"),
    (lambda o, l, i: o.dora_policy_loss(l, l, l, dual_clip=0.5), "DORA_ERR_FLAGS"),
    (lambda o, l, i: o.dora_policy_loss(l, l, l, denominator=0), "more than 0"),
    (lambda o, l, i: o.dora_policy_loss(l, l, l, reduce="mean"), "expected one of"),
    (lambda o, l, i: o.dora_policy_loss(l, l.cpu(), l), "device"),
    (lambda o, l, i: o.dora_policy_loss_backward(l[0], l[0, :1], l, l, l), "one number"),
])
def test_refusals(ops, call, message):
    l, i = torch.zeros(4, 6, device="cuda"), torch.tensor([0, 1], device="cuda")
    with pytest.raises((ValueError, TypeError, RuntimeError), match=message):
        call(ops, l, i)
