"""The optimizer's bookkeeping on the host: which plans it keeps, what its state follows.  The
operators are replaced by a recorder, so no GPU is needed."""
from __future__ import annotations

import copy
import pickle

import pytest
import torch

from parameter_efficient_fine_dora_amd import _lib, ops, optim


class Plan:
    """Notes the addresses of a step's tensors, as ops.AdamWPlan does."""
    made = []

    def __init__(self, params, exp_avg, exp_avg_sq, **more):
        self.params = list(params)
        self.lists = [self.params, list(exp_avg), list(exp_avg_sq)]
        self.lists += [list(v) for v in more.values() if v is not None]
        self.more = {k: v for k, v in more.items() if v is not None}
        self.table = (_lib.DoraAdamwTensor * len(self.params))()
        for e, p in zip(self.table, self.params):
            e.param = p.data_ptr()
        self.addresses = self.where()
        Plan.made.append(self)

    def where(self):
        return [[t.data_ptr() for t in lst] for lst in self.lists]

    def unchanged(self):
        return self.addresses == self.where()


@pytest.fixture(autouse=True)
def recorder(monkeypatch):
    """Steps as (plan, step, parameters) instead of launches."""
    steps = []
    Plan.made = []
    monkeypatch.setattr(ops, "AdamWPlan", Plan)
    monkeypatch.setattr(ops, "dora_adamw", lambda plan, grads, **kw: steps.append((plan, kw)))
    monkeypatch.setattr(ops, "dora_grad_norm", lambda plan, grads, most: (torch.tensor(1.0),) * 2)
    return steps


def params(*sizes, dtype=torch.bfloat16):
    out = [torch.nn.Parameter(torch.randn(n).to(dtype)) for n in sizes]
    for p in out:
        p.grad = torch.ones_like(p)
    return out


@pytest.mark.parametrize("bits", [32, 8])
def test_a_state_whose_storage_was_exchanged_makes_the_plan_anew(recorder, bits):
    """What moving states to the host and back does: the tensor objects stay, their memory does not."""
    ps = params(300, 5)
    opt = optim.AdamW(ps, state_bits=bits, master=True)
    opt.step()
    opt.step()
    assert len(Plan.made) == 1                       # kept while nothing changes
    made = 1
    for name in [k for k in opt.state[ps[0]] if k != "step"]:
        state = opt.state[ps[0]]
        state[name].data = state[name].data.clone()
        opt.step()
        made += 1
        assert len(Plan.made) == made, name
        plan = recorder[-1][0]
        assert any(state[name] is t for lst in plan.lists for t in lst)
        assert plan.unchanged()


@pytest.mark.parametrize("how", ["deepcopy", "pickle"])
def test_a_copy_steps_as_the_original(recorder, how):
    """torch keeps an optimizer's defaults, state and groups alone; the options have to come along."""
    ps = params(300, 5)
    opt = optim.AdamW(ps, state_bits=8, master=True, max_norm=0.5)
    opt.step()
    twin = copy.deepcopy(opt) if how == "deepcopy" else pickle.loads(pickle.dumps(opt))
    assert (twin.state_bits, twin.master, twin.max_norm) == (8, True, 0.5)
    mine = twin.param_groups[0]["params"]
    assert all(a is not b and torch.equal(a, b) for a, b in zip(mine, ps))
    for p in mine:
        p.grad = torch.ones_like(p)
    twin.step()
    plan, kw = recorder[-1]
    assert all(a is b for a, b in zip(plan.params, mine)) and kw["step"] == 2
    assert set(plan.more) == {"masters", "exp_avg_scales", "exp_avg_sq_scales"}
    assert opt.state[ps[0]]["step"] == 1


def checkpoint(ps, cls=torch.optim.AdamW, **kw):
    twins = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    for p in twins:
        p.grad = torch.ones_like(p)
    opt = cls(twins, lr=1e-3, **kw)
    for _ in range(3):
        opt.step()
    return opt.state_dict()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_torchs_checkpoint_keeps_one_call_for_a_group(recorder, dtype):
    """Its step counts are tensors, one per parameter, and its moments have the parameters' type."""
    ps = params(300, 5, dtype=dtype)
    opt = optim.AdamW(ps)
    saved = checkpoint(ps)
    opt.load_state_dict(saved)
    for p, s in zip(ps, saved["state"].values()):
        mine = opt.state[p]
        assert type(mine["step"]) is int and mine["step"] == 3
        for k in ("exp_avg", "exp_avg_sq"):
            assert mine[k].dtype == torch.float32 and torch.equal(mine[k], s[k].float())
    opt.step()
    assert len(recorder) == 1 and recorder[0][1]["step"] == 4 and len(recorder[0][0].params) == 2


@pytest.mark.parametrize("cls,kw,word", [
    (torch.optim.AdamW, dict(amsgrad=True), "amsgrad"), (torch.optim.AdamW, dict(maximize=True), "maximize"),
    (torch.optim.Adam, dict(weight_decay=0.1), "decoupled")])
def test_a_checkpoint_of_another_update_is_refused(cls, kw, word):
    ps = params(30)
    opt = optim.AdamW(ps, lr=0.5)
    with pytest.raises(ValueError, match=word):
        opt.load_state_dict(checkpoint(ps, cls, **kw))
    assert not opt.state and opt.param_groups[0]["lr"] == 0.5
    opt.load_state_dict(checkpoint(ps, torch.optim.Adam))       # without decay it is the same update
    assert opt.state[ps[0]]["step"] == 3


@pytest.mark.parametrize("saved,bits", [(32, 8), (8, 32)])
def test_moments_of_the_other_width_are_refused_by_name(recorder, saved, bits):
    ps = params(300, 5)
    other = optim.AdamW(ps, state_bits=saved)
    other.step()
    opt = optim.AdamW(ps, state_bits=bits, lr=0.5)
    with pytest.raises(ValueError, match=f"moments of {saved} bits.*state_bits={bits}"):
        opt.load_state_dict(other.state_dict())
    assert not opt.state and opt.param_groups[0]["lr"] == 0.5
    opt.step()


def test_moments_that_are_incomplete_are_refused(recorder):
    ps = params(300, 5)
    opt = optim.AdamW(ps, state_bits=8)
    opt.step()
    saved = copy.deepcopy(opt.state_dict())
    del saved["state"][1]["exp_avg_sq_scale"]
    with pytest.raises(ValueError, match="exp_avg_sq_scale"):
        optim.AdamW(ps, state_bits=8).load_state_dict(saved)
    with pytest.raises(ValueError, match="exp_avg"):
        optim.AdamW(ps).load_state_dict(torch.optim.SGD(ps, lr=0.1, momentum=0.9).state_dict()
                                        | dict(state={0: dict(momentum_buffer=torch.ones(300))}))


def test_masters_follow_the_option_and_not_the_checkpoint(recorder):
    """Made from the parameters where the checkpoint has none, left out where they are not wanted."""
    for saved, wanted in ((False, True), (True, False), (True, True)):
        ps = params(300, 5)
        other = optim.AdamW(ps, master=saved)
        other.step()
        opt = optim.AdamW(ps, master=wanted)
        opt.load_state_dict(other.state_dict())
        opt.step()
        plan = recorder[-1][0]
        assert ("masters" in plan.more) == wanted
        assert all(("master" in opt.state[p]) == wanted for p in ps)
        if wanted:
            for p, w in zip(ps, plan.more["masters"]):
                assert w.dtype == torch.float32 and torch.equal(w, p.detach().float())


def test_a_parameter_without_a_master_among_others_that_have_one(recorder):
    """One joins after a checkpoint was loaded; the plan of the norm takes both."""
    ps = params(300, 5)
    saved = optim.AdamW(ps)
    saved.step()
    state = copy.deepcopy(saved.state_dict())
    del state["state"][0]
    opt = optim.AdamW(ps, master=True, max_norm=1.0)
    opt.load_state_dict(state)
    opt.step()
    assert all(len(p.more["masters"]) == len(p.params) for p in Plan.made if "masters" in p.more)
    assert [set(opt.state[p]) for p in ps] == [{"step", "exp_avg", "exp_avg_sq", "master"}] * 2


def test_a_master_goes_with_its_parameters_type(recorder):
    p, = params(300)
    opt = optim.AdamW([p], master=True)
    opt.step()
    for dtype in (torch.float32, torch.bfloat16):
        p.grad = None
        p.data = torch.randn(300).to(dtype)
        p.grad = torch.ones_like(p)
        opt.step()
        assert ("masters" in recorder[-1][0].more) == (dtype == torch.bfloat16)
    assert torch.equal(opt.state[p]["master"], p.detach().float())
