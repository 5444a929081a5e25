"""Measured cases of the operators that preference and policy fine-tuning adds to a step.

Training on preferences turns the log probabilities of two answers' tokens (and a frozen
reference's) into a paired loss; training on rewards turns them into a clipped policy loss with a
divergence from the reference.  Both send a gradient back to the token log probabilities.  The
update of an adapter's matrices may then be orthogonalised by Newton-Schulz products before it is
applied (Muon).

``own`` False: plain elementary torch operations, rounded once at the end.  ``own`` True: the
package's operators.  ``exact`` is the definition in float64.
"""
from __future__ import annotations

import functools
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
COEFFICIENTS = ((3.4445, -4.7750, 2.0315),) * 5
NS_EPS = 1e-7
BETA, MARGIN, SMOOTHING = 0.1, 0.0, 0.05
CLIP_LOW, CLIP_HIGH, DUAL, KL_COEF = 0.2, 0.28, 3.0, 0.05
LR, MOMENTUM, DECAY = 2e-3, 0.95, 0.01


# ---- cases ------------------------------------------------------------------------

def listed():
    return [
        # one pair of answers scored: latency only
        dict(name="preference_one_pair", op="preference", way="forward", sequences=2, length=512,
             packed=False, ref=True, kind="sigmoid", normalize=False),
        # a training batch of packed answers of different lengths, loss and gradient
        dict(name="preference_packed", op="preference", way="train", sequences=254, length=1031,
             packed=True, ref=True, kind="sigmoid", normalize=True),
        # long padded answers without a reference, the gradient alone
        dict(name="preference_long_backward", op="preference", way="backward", sequences=128,
             length=32768, packed=False, ref=False, kind="square", normalize=False),
        # a few short answers of one prompt, loss and gradient: latency
        dict(name="policy_one_group", op="policy", way="train", sequences=8, length=256,
             packed=False, ref=True, advantage="sequence", reduce="token", dual=False),
        # a step's answers packed, one advantage each, every answer of the same weight
        dict(name="policy_packed", op="policy", way="train", sequences=512, length=2011,
             packed=True, ref=True, advantage="sequence", reduce="sequence", dual=False),
        # the loss of an odd padded batch without a reference
        dict(name="policy_odd_forward", op="policy", way="forward", sequences=61, length=4099,
             packed=False, ref=False, advantage="token", reduce="token", dual=False),
        # the largest batch's gradient, advantages per token, both sides of the ratio bounded
        dict(name="policy_long_backward", op="policy", way="backward", sequences=256, length=16384,
             packed=False, ref=True, advantage="token", reduce="token", dual=True),
        # the momentum of one rank-64 adapter
        dict(name="orthogonalize_rank64", op="orthogonalize", count=1, rows=64, cols=2048,
             dtype="bf16"),
        # a float32 matrix of odd sizes, taller than wide
        dict(name="orthogonalize_odd", op="orthogonalize", count=1, rows=1031, cols=517, dtype="f32"),
        # the whole weight of a 2048 x 6144 layer
        dict(name="orthogonalize_weight", op="orthogonalize", count=1, rows=2048, cols=6144,
             dtype="bf16"),
        # a step on the adapters of 24 high-rank layers
        dict(name="muon_adapters", op="muon", layers=24, d_out=8192, d_in=8192, r=384, dtype="bf16",
             master=False),
        # a step on the adapters of 56 rank-64 layers with float32 masters
        dict(name="muon_master", op="muon", layers=56, d_out=2048, d_in=6144, r=64, dtype="bf16",
             master=True),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi], odd ones as likely as even ones."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["preference", "policy", "orthogonalize", "muon"])
    if op in ("preference", "policy"):
        sequences = _spread(rng, 1, 512) * 2
        length = _spread(rng, 1, min(65536, 4194304 // sequences))
        case = dict(op=op, way=rng.choice(["forward", "backward", "train", "train"]),
                    sequences=sequences, length=length, packed=rng.random() < 0.5,
                    ref=rng.random() < 0.7)
        if op == "preference":
            return dict(case, kind=rng.choice(["sigmoid", "hinge", "square"]),
                        normalize=rng.random() < 0.4)
        return dict(case, advantage=rng.choice(["sequence", "token"]),
                    reduce=rng.choice(["sequence", "token"]), dual=rng.random() < 0.3)
    if op == "orthogonalize":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        n = _spread(rng, 4, 2048 if dtype == "bf16" else 1100)
        m = _spread(rng, n, min(27648, max(n, 25769803776 // (n * n))))
        count = _spread(rng, 1, max(1, min(64, 33554432 // (n * m))))
        rows, cols = (n, m) if rng.random() < 0.5 else (m, n)
        return dict(op=op, count=count, rows=rows, cols=cols, dtype=dtype)
    d_out, d_in, r = _spread(rng, 64, 8192), _spread(rng, 64, 8192), _spread(rng, 4, 384)
    if rng.random() < 0.5:
        d_out, d_in, r = (d_out + 7) // 8 * 8, (d_in + 7) // 8 * 8, (r + 7) // 8 * 8
    layers = _spread(rng, 1, max(1, min(64, 24 * 6291456 // (2 * (d_out + d_in) * r))))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    return dict(op="muon", layers=layers, d_out=d_out, d_in=d_in, r=r, dtype=dtype,
                master=dtype == "bf16" and rng.random() < 0.5)


# ---- inputs -----------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _sequences(case, g):
    """Token log probabilities of sequences: the policy's, and which tokens count."""
    S, L = case["sequences"], case["length"]
    at = torch.arange(S * L, device="cuda")
    # an answer's length: from a few tokens to twice the mean, or a padded row's used part
    share = 0.05 + 0.9 * torch.rand(S, device="cuda", generator=g)
    if case["packed"]:
        lengths = (2 * L * share).long().clamp_(min=1)
        offsets = torch.zeros(S + 1, dtype=torch.int64, device="cuda")
        torch.cumsum(lengths, 0, out=offsets[1:])
        offsets = (offsets * (S * L) // offsets[-1]).contiguous()   # the batch's budget is filled
        row = torch.searchsorted(offsets, at, right=True) - 1
        column, ends = at - offsets[row], offsets[1:] - offsets[:-1]
    else:
        offsets = None
        row, column, ends = at // L, at % L, (L * (0.3 + 0.7 * share)).long().clamp_(min=1)
    shape = (S * L,) if case["packed"] else (S, L)
    prompt = (ends * 0.2 * torch.rand(S, device="cuda", generator=g)).long()
    mask = (column >= prompt[row]) & (column < ends[row])
    # most tokens are near certain, a few are surprising
    logp = -3.0 * torch.rand(S * L, device="cuda", generator=g) ** 3 - 0.01
    logp = torch.where(mask, logp, 0.0)

    def other(scale):
        step = scale * torch.randn(S * L, device="cuda", generator=g)
        return torch.where(mask, (logp + step).clamp(max=-1e-4), 0.0).view(shape)

    return dict(logp=logp.view(shape), mask=mask.view(shape), offsets=offsets), other


def _prepare_preference(case, g):
    s, other = _sequences(case, g)
    S = case["sequences"]
    P = S // 2
    order = torch.randperm(S, device="cuda", generator=g)
    # answers 2p and 2p + 1 of a shuffled batch, and a quarter of the pairs shares the first's
    chosen, rejected = order[0::2].clone(), order[1::2].clone()
    chosen[:P // 4] = chosen[0].clone()
    s.update(op="preference", way=case["way"], ref=other(0.05) if case["ref"] else None,
             chosen=chosen, rejected=rejected, kind=case["kind"], normalize=case["normalize"],
             grad=torch.full((P,), 1.0 / P, device="cuda"))
    if case["way"] == "backward":
        loss, score, logit, count = _preference_forward(s)
        s.update(logit=logit, count=count)
    return s


def _prepare_policy(case, g):
    s, other = _sequences(case, g)
    S = case["sequences"]
    adv = torch.randn(S if case["advantage"] == "sequence" else s["logp"].shape, device="cuda",
                      generator=g)
    s.update(op="policy", way=case["way"], old=other(0.1), ref=other(0.2) if case["ref"] else None,
             advantages=adv, reduce=case["reduce"], dual=DUAL if case["dual"] else None,
             grad=torch.ones((), device="cuda"))
    if case["way"] == "backward":
        s["weight"] = _policy_forward(s)[2]
    return s


def _matrices(count, rows, cols, g):
    """Gradients: a few strong directions over a floor of noise."""
    k = min(rows, cols, 32)
    left = torch.randn(count, rows, k, device="cuda", generator=g)
    right = torch.randn(count, k, cols, device="cuda", generator=g)
    left *= torch.logspace(0, -1, k, device="cuda") / math.sqrt(k)
    return torch.bmm(left, right).add_(torch.randn(count, rows, cols, device="cuda", generator=g),
                                       alpha=0.3)


def _prepare_orthogonalize(case, g):
    x = _matrices(case["count"], case["rows"], case["cols"], g).to(DTYPES[case["dtype"]])
    return dict(op="orthogonalize", x=x)


def _prepare_muon(case, g):
    n, r, dt = case["layers"], case["r"], DTYPES[case["dtype"]]
    shapes = ((r, case["d_in"]), (case["d_out"], r))
    params, grads, momenta = [], [], []
    for rows, cols in shapes:
        std = 1.0 / math.sqrt(3.0 * cols) if rows == r else 0.01
        params.append((std * torch.randn(n, rows, cols, device="cuda", generator=g)).to(dt))
        grads.append((1e-3 * _matrices(n, rows, cols, g)).to(dt))
        momenta.append(1e-3 * _matrices(n, rows, cols, g))
    masters = [p.float() for p in params] if case["master"] else None
    # a program keeps one tensor a layer; they lie side by side so that they come back whole
    state = dict(op="muon", params=params, grads=grads, momenta=momenta, masters=masters)

    def each(stacks):
        return [t for stack in stacks for t in stack.unbind(0)]

    state["lists"] = (each(params), each(grads), each(momenta), each(masters) if masters else None)
    return state


def prepare(case, seed):
    return globals()["_prepare_" + case["op"]](case, _generator(seed))


# ---- plain forms ------------------------------------------------------------------

def _sums(values, s):
    """Sums of values [..] (float64) over each sequence, float64 [S]."""
    if s["offsets"] is None:
        return values.sum(1)
    run = torch.nn.functional.pad(torch.cumsum(values, 0), (1, 0))
    return run[s["offsets"][1:]] - run[s["offsets"][:-1]]


def _over_tokens(values, s):
    """values [S] spread over each sequence's tokens."""
    if s["offsets"] is None:
        return values[:, None].expand(s["logp"].shape)
    at = torch.arange(s["logp"].numel(), device="cuda")
    return values[torch.searchsorted(s["offsets"], at, right=True) - 1]


def _preference_forward(s):
    """(loss, score, logit, count): sums over thousands of tokens, so in 64 bits."""
    r = s["logp"].double()
    if s["ref"] is not None:
        r = r - s["ref"].double()
    total = _sums(torch.where(s["mask"], r, 0.0), s)
    count = _sums(s["mask"].double(), s)
    if s["normalize"]:
        total = total / count.clamp(min=1.0)
    score = BETA * total
    h = score[s["chosen"]] - score[s["rejected"]] - MARGIN
    if s["kind"] == "sigmoid":
        loss = (1.0 - SMOOTHING) * _softplus(-h) + SMOOTHING * _softplus(h)
    elif s["kind"] == "hinge":
        loss = (1.0 - h).clamp(min=0.0)
    else:
        loss = ((h - 0.5) / BETA) ** 2
    return loss.float(), score.float(), h.float(), count.float()


def _softplus(v):
    return v.clamp(min=0.0) + torch.log1p(torch.exp(-v.abs()))


def _preference_backward(s, h, count):
    h = h.double()
    if s["kind"] == "sigmoid":
        slope = SMOOTHING - 1.0 / (1.0 + torch.exp(h))
    elif s["kind"] == "hinge":
        slope = torch.where(h < 1.0, -1.0, 0.0).double()
    else:
        slope = 2.0 * (h - 0.5) / BETA ** 2
    each = BETA * slope * s["grad"]
    per = torch.zeros(count.numel(), dtype=torch.float64, device="cuda")
    per = per.index_add(0, s["chosen"], each).index_add(0, s["rejected"], -each)
    if s["normalize"]:
        per = per / count.double().clamp(min=1.0)
    return torch.where(s["mask"], _over_tokens(per, s), 0.0).float()


def _policy_terms(s):
    """Per token in 64 bits (a ratio beside its bound must fall on the right side): the loss, its
    slope in logp, the divergence, whether the bound holds it, the ratio."""
    logp = s["logp"].double()
    ratio = torch.exp(logp - s["old"].double())
    adv = s["advantages"].double()
    if adv.shape != logp.shape:
        adv = _over_tokens(adv, s)
    clipped = ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    gain = torch.minimum(ratio * adv, clipped * adv)
    held = ratio * adv > clipped * adv
    if s["dual"] is not None:
        low = s["dual"] * adv
        lower = (adv < 0.0) & (gain < low)
        gain = torch.where(lower, low, gain)
        held = held | lower
    loss, slope = -gain, torch.where(held, 0.0, -ratio * adv)
    kl = torch.zeros_like(loss)
    if s["ref"] is not None:
        d = s["ref"].double() - logp
        kl = torch.expm1(d) - d
        loss = loss + KL_COEF * kl
        slope = slope - KL_COEF * torch.expm1(d)
    return loss, slope, kl, held.double(), ratio


def _policy_forward(s):
    """(loss, stats, weight): weight is each sequence's factor on its tokens, or one for all."""
    loss, _, kl, held, ratio = (torch.where(s["mask"], t, 0.0) for t in _policy_terms(s))
    total = s["mask"].double().sum()
    if s["reduce"] == "sequence":
        count = _sums(s["mask"].double(), s)
        live = (count > 0).double().sum()
        weight = torch.where(count > 0, 1.0 / (count.clamp(min=1.0) * live.clamp(min=1.0)), 0.0)
        value = (_sums(loss, s) * weight).sum()
    else:
        weight = (1.0 / total.clamp(min=1.0)).view(1)
        value = loss.sum() * weight[0]
    means = [t.sum() / total.clamp(min=1.0) for t in (kl, held, ratio)]
    return value.float(), torch.stack([*means, total]).float(), weight.float()


def _policy_backward(s, weight):
    slope = _policy_terms(s)[1]
    weight = weight.double()
    if s["reduce"] == "sequence":
        weight = _over_tokens(weight, s)
    return torch.where(s["mask"], s["grad"] * weight * slope, 0.0).float()


def _newton_schulz(x):
    """The plain iteration in float32 on a stack of matrices."""
    flip = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2).contiguous() if flip else x
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt().float()

    def step(x, abc):
        a, b, c = abc
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        return a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)

    x = functools.reduce(step, COEFFICIENTS, x / (norm + NS_EPS))
    return x.transpose(1, 2) if flip else x


def _update_scale(rows, cols):
    return 0.2 * math.sqrt(max(rows, cols))


def _muon_stack(param, grad, momentum, master):
    """One step on a stack of matrices, in place."""
    g = grad.float()
    momentum.lerp_(g, 1.0 - MOMENTUM)
    update = _newton_schulz((1.0 - MOMENTUM) * g + MOMENTUM * momentum)
    p = param.float() if master is None else master
    p = p * (1.0 - LR * DECAY) - LR * _update_scale(*param.shape[1:]) * update
    if master is not None:
        master.copy_(p)
    param.copy_(p)


# ---- a pass -----------------------------------------------------------------------

def _own_preference(s):
    from parameter_efficient_fine_dora_amd import ops
    how = dict(kind=s["kind"], beta=BETA, margin=MARGIN, smoothing=SMOOTHING,
               normalize=s["normalize"], mask=s["mask"], offsets=s["offsets"])
    if s["way"] == "backward":
        logit, count = s["logit"], s["count"]
    else:
        loss, score, logit, count = ops.dora_preference_loss(s["logp"], s["chosen"], s["rejected"],
                                                             ref_logp=s["ref"], **how)
        if s["way"] == "forward":
            return loss, score
    grad = ops.dora_preference_loss_backward(s["grad"], logit, count, s["chosen"], s["rejected"],
                                             shape=s["logp"].shape, **how)
    return grad if s["way"] == "backward" else (loss, score, grad)


def _own_policy(s):
    from parameter_efficient_fine_dora_amd import ops
    how = dict(ref_logp=s["ref"], mask=s["mask"], offsets=s["offsets"], clip=(CLIP_LOW, CLIP_HIGH),
               dual_clip=s["dual"], kl_coef=KL_COEF if s["ref"] is not None else 0.0,
               reduce=s["reduce"])
    if s["way"] == "backward":
        weight = s["weight"]
    else:
        loss, stats, weight = ops.dora_policy_loss(s["logp"], s["old"], s["advantages"], **how)
        if s["way"] == "forward":
            return loss, stats
    grad = ops.dora_policy_loss_backward(s["grad"], weight, s["logp"], s["old"], s["advantages"],
                                         **how)
    return grad if s["way"] == "backward" else (loss, stats, grad)


def _own_muon(s):
    from parameter_efficient_fine_dora_amd import ops
    params, grads, momenta, masters = s["lists"]
    plan = s.get("plan")
    if plan is None:
        plan = s["plan"] = ops.MuonPlan(params, momenta, masters=masters)
    ops.dora_muon(plan, grads, lr=LR, momentum=MOMENTUM, nesterov=True, weight_decay=DECAY,
                  coefficients=COEFFICIENTS, eps=NS_EPS, adjust="rms")


def _run_preference(s):
    if own:
        return _own_preference(s)
    if s["way"] == "backward":
        return _preference_backward(s, s["logit"], s["count"])
    loss, score, logit, count = _preference_forward(s)
    if s["way"] == "forward":
        return loss, score
    return loss, score, _preference_backward(s, logit, count)


def _run_policy(s):
    if own:
        return _own_policy(s)
    if s["way"] == "backward":
        return _policy_backward(s, s["weight"])
    loss, stats, weight = _policy_forward(s)
    return (loss, stats) if s["way"] == "forward" else (loss, stats, _policy_backward(s, weight))


def _run_orthogonalize(s):
    if own:
        from parameter_efficient_fine_dora_amd import ops
        return ops.dora_orthogonalize(s["x"], coefficients=COEFFICIENTS, eps=NS_EPS)
    return _newton_schulz(s["x"].float()).to(s["x"].dtype).contiguous()


def _run_muon(s):
    if own:
        _own_muon(s)
    else:
        masters = s["masters"] or (None, None)
        _muon_stack(s["params"][0], s["grads"][0], s["momenta"][0], masters[0])
        _muon_stack(s["params"][1], s["grads"][1], s["momenta"][1], masters[1])
    return dict(params=s["params"], momenta=s["momenta"], masters=s["masters"])


def run(state):
    return globals()["_run_" + state["op"]](state)


def work(case):
    op = case["op"]
    if op in ("preference", "policy"):
        n, S = case["sequences"] * case["length"], case["sequences"]
        ways = {"forward": (1, 0), "backward": (0, 1), "train": (1, 1)}[case["way"]]
        offsets = 8 * (S + 1) if case["packed"] else 0
        if op == "preference":
            # forward: log probabilities, the reference's, the mask; backward: mask and gradient
            forward = n * (5 + 4 * case["ref"]) + S // 2 * 24 + S * 8 + offsets
            backward = n * 5 + S // 2 * 24 + S * 4 + offsets
            return dict(bytes=ways[0] * forward + ways[1] * backward, flops=n * (3 * ways[0] + ways[1]))
        adv = 4 * (n if case["advantage"] == "token" else S)
        read = n * (9 + 4 * case["ref"]) + adv + offsets
        return dict(bytes=sum(ways) * read + ways[1] * 4 * n, flops=20 * n * sum(ways))
    if op == "orthogonalize":
        shapes = [(case["rows"], case["cols"], case["count"])]
        per = 2 * (2 if case["dtype"] == "bf16" else 4)
    else:
        shapes = [(case["r"], case["d_in"], case["layers"]), (case["d_out"], case["r"], case["layers"])]
        size = 2 if case["dtype"] == "bf16" else 4
        per = size + 8 + (8 + size if case["master"] else 2 * size)
    # X X^T (half of it), one product of X with the polynomial of that, and the polynomial's own
    # products of symmetric matrices: one for the first step, four for each other, one fewer twice
    flops = sum(k * (3 * min(a, b) ** 2 * max(a, b) + 17 * min(a, b) ** 3) for a, b, k in shapes)
    return dict(bytes=sum(a * b * k for a, b, k in shapes) * per, flops=flops)


# ---- the definition in 64 bits ------------------------------------------------------

def _spans(s):
    if s["offsets"] is None:
        S, L = s["logp"].shape
        return [(i * L, (i + 1) * L) for i in range(S)]
    o = s["offsets"].tolist()
    return list(zip(o, o[1:]))


def _flat(t):
    return None if t is None else t.double().reshape(-1)


def _exact_preference(s):
    logp, ref, mask = _flat(s["logp"]), _flat(s["ref"]), s["mask"].reshape(-1)
    spans = _spans(s)
    score = torch.zeros(len(spans), dtype=torch.float64, device="cuda")
    count = torch.zeros_like(score)
    for i, (a, b) in enumerate(spans):
        live = mask[a:b]
        v = logp[a:b][live] if ref is None else (logp[a:b] - ref[a:b])[live]
        count[i] = v.numel()
        score[i] = BETA * (v.mean() if s["normalize"] and v.numel() else v.sum())
    h = (score[s["chosen"]] - score[s["rejected"]] - MARGIN).requires_grad_()
    if s["kind"] == "sigmoid":
        both = torch.nn.functional.logsigmoid(torch.stack([h, -h]))
        loss = -(1.0 - SMOOTHING) * both[0] - SMOOTHING * both[1]
    elif s["kind"] == "hinge":
        loss = torch.nn.functional.relu(1.0 - h)
    else:
        loss = (h / BETA - 0.5 / BETA) ** 2
    if s["way"] == "forward":
        return loss.detach(), score
    if s["way"] == "backward":       # from the logits that the state holds
        with torch.no_grad():
            h.copy_(s["logit"])
        loss = {"sigmoid": lambda: -(1.0 - SMOOTHING) * torch.nn.functional.logsigmoid(h)
                - SMOOTHING * torch.nn.functional.logsigmoid(-h),
                "hinge": lambda: torch.nn.functional.relu(1.0 - h),
                "square": lambda: (h / BETA - 0.5 / BETA) ** 2}[s["kind"]]()
    slope, = torch.autograd.grad((loss * s["grad"].double()).sum(), h)
    chosen, rejected = s["chosen"].tolist(), s["rejected"].tolist()
    per = [0.0] * len(spans)
    for c, w, v in zip(chosen, rejected, (BETA * slope).tolist()):
        per[c] += v
        per[w] -= v
    grad = torch.zeros_like(logp)
    counts = count.tolist()
    for i, (a, b) in enumerate(spans):
        grad[a:b] = per[i] / (max(counts[i], 1.0) if s["normalize"] else 1.0)
    grad = (grad * mask).view(s["logp"].shape)
    return grad if s["way"] == "backward" else (loss.detach(), score, grad)


def _exact_policy(s):
    mask = s["mask"].reshape(-1)
    spans = _spans(s)
    adv = _flat(s["advantages"])
    if s["advantages"].shape != s["logp"].shape:
        per = adv.tolist()
        adv = torch.empty(mask.numel(), dtype=torch.float64, device="cuda")
        for i, (a, b) in enumerate(spans):
            adv[a:b] = per[i]
    live = mask.nonzero().flatten()
    x = _flat(s["logp"])[live].requires_grad_()
    ratio = torch.exp(x - _flat(s["old"])[live])
    a = adv[live]
    # a gain grows with the ratio only up to the bound that its sign sets
    top = torch.full_like(a, math.inf if s["dual"] is None else s["dual"])
    bottom = torch.full_like(a, 1.0 - CLIP_LOW)
    top[a >= 0] = 1.0 + CLIP_HIGH
    bottom[a >= 0] = 0.0
    inside = (ratio <= top) & (ratio >= bottom)
    loss = -a * torch.where(inside, ratio, torch.where(ratio > top, top, bottom).detach())
    kl = torch.zeros_like(loss)
    if s["ref"] is not None:
        d = _flat(s["ref"])[live] - x
        kl = torch.special.expm1(d) - d
        loss = loss + KL_COEF * kl
    n = live.numel()
    if s["reduce"] == "sequence":
        counts = [int(mask[p:q].sum()) for p, q in spans]
        some = max(1, sum(c > 0 for c in counts))
        weight = torch.zeros(mask.numel(), dtype=torch.float64, device="cuda")
        for c, (p, q) in zip(counts, spans):
            weight[p:q] = 1.0 / (max(c, 1) * some)
        weight = weight[live]
    else:
        weight = torch.full((n,), 1.0 / max(n, 1), dtype=torch.float64, device="cuda")
    value = (loss * weight).sum()
    if s["way"] != "forward":
        g, = torch.autograd.grad(value, x)
        grad = torch.zeros(mask.numel(), dtype=torch.float64, device="cuda")
        grad[live] = g
        grad = grad.view(s["logp"].shape)
        if s["way"] == "backward":
            return grad
    held = a.new_tensor([float((~inside).double().mean()) if n else 0.0])
    stats = torch.stack([kl.detach().mean(), held[0], ratio.detach().mean(),
                         a.new_tensor(float(n))]) if n else torch.zeros(4, dtype=torch.float64)
    return (value.detach(), stats) if s["way"] == "forward" else (value.detach(), stats, grad)


def _exact_polynomial(x):
    """One matrix in float64, a row-vector at a time of the shorter side: X <- (a + b S + c S^2) X."""
    x = x.double()
    x = x / (torch.linalg.matrix_norm(x) + NS_EPS)
    for a, b, c in COEFFICIENTS:
        if x.shape[0] <= x.shape[1]:
            s = x @ x.mT
            x = a * x + b * (s @ x) + c * (s @ (s @ x))
        else:
            s = x.mT @ x
            x = a * x + b * (x @ s) + c * ((x @ s) @ s)
    return x


def _exact_muon(s):
    params, momenta, masters = [], [], []
    for k in range(2):
        g = s["grads"][k].double()
        m = MOMENTUM * s["momenta"][k].double() + (1.0 - MOMENTUM) * g
        momenta.append(m)
        p = (s["masters"] or s["params"])[k].double()
        rate = LR * _update_scale(*p.shape[1:])
        out = torch.empty_like(p)
        for i in range(p.shape[0]):
            u = MOMENTUM * m[i] + (1.0 - MOMENTUM) * g[i]
            out[i] = p[i] - LR * DECAY * p[i] - rate * _exact_polynomial(u)
        params.append(out)
        masters.append(out)
    return dict(params=params, momenta=momenta, masters=masters if s["masters"] else None)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "preference":
        return _exact_preference(s)
    if case["op"] == "policy":
        return _exact_policy(s)
    if case["op"] == "orthogonalize":
        return torch.stack([_exact_polynomial(x) for x in s["x"]])
    return _exact_muon(s)
