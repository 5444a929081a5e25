"""Muon's bookkeeping on the host: plans on tensors that are only looked at, the compiled step replaced by
a recorder, so that no GPU is needed."""
from __future__ import annotations

import ctypes
import math
import os

import pytest
import torch

from parameter_efficient_fine_dora_amd import _lib, ops, optim

pytestmark = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="libdora.so not built")


class Recorder:
    """The compiled entry points: notes the workspace that a step got, and refuses what the library's
    size says is refused."""

    def __init__(self):
        self.steps = []

    def muon_grads(self, *args):
        return None

    def muon_step(self, table, params, how, ws, ws_bytes, stream):
        options = _lib.DoraMuonOptions.from_address(how)
        entries = (_lib.DoraMuonTensor * len(params)).from_address(table)
        need = _lib.lib().dora_muon_workspace_bytes(entries, len(params), ctypes.byref(options))
        self.steps.append((ws_bytes, need))
        if not need:
            return _lib.ERR_CODE["DORA_ERR_FLAGS"]
        return _lib.ERR_CODE["DORA_ERR_WORKSPACE"] if ws_bytes < need else 0


@pytest.fixture
def compiled(monkeypatch):
    """Host tensors pass for device tensors, and the recorder for the compiled module."""
    def need(t, name, dtype=None, shape=None, dev=None):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t

    recorder = Recorder()
    monkeypatch.setattr(ops, "_need", need)
    monkeypatch.setattr(ops, "_compiled", lambda: recorder)
    monkeypatch.setattr(ops, "_stream", lambda dev: 0)
    monkeypatch.setattr(ops, "_given_ws", lambda ws, dev: ws.numel())
    return recorder


def plan_of(*sizes, dtype=torch.float32):
    params = [torch.ones(*s, dtype=dtype) for s in sizes]
    return ops.MuonPlan(params, [torch.zeros(*s) for s in sizes]), [torch.ones(*s, dtype=dtype) for s in sizes]


@pytest.mark.parametrize("bad", [dict(lr=math.nan), dict(lr=math.inf), dict(momentum=1.0), dict(momentum=-0.5),
                                 dict(eps=0.0), dict(weight_decay=math.inf)], ids=str)
def test_a_refused_step_spoils_no_later_one(compiled, bad):
    plan, grads = plan_of((256, 1024))
    with pytest.raises(_lib.DoraError, match="DORA_ERR_FLAGS"):
        ops.dora_muon(plan, grads, **dict(dict(lr=0.1), **bad))
    for _ in range(2):
        ops.dora_muon(plan, grads, lr=0.1)
    assert compiled.steps[-1][0] >= compiled.steps[-1][1] > 0


def test_other_coefficients_get_their_own_workspace(compiled):
    plan, grads = plan_of((256, 1024))
    for steps in (5, 16, 1, 5):
        ops.dora_muon(plan, grads, lr=0.1, coefficients=((3.4445, -4.7750, 2.0315),) * steps)
        got, need = compiled.steps[-1]
        assert got == need > 0


def parameters():
    return [torch.nn.Parameter(torch.ones(6, 8)), torch.nn.Parameter(torch.ones(8, 6))]


def others():
    """Optimizers whose state has a momentum_buffer too."""
    yield torch.optim.SGD, dict(lr=0.1, momentum=0.9), "eps"
    if hasattr(torch.optim, "Muon"):
        yield torch.optim.Muon, dict(lr=0.1), "coefficients"


@pytest.mark.parametrize("kind,how,lacks", list(others()), ids=lambda v: getattr(v, "__name__", None))
def test_another_optimizers_checkpoint_is_refused(kind, how, lacks):
    theirs = parameters()
    other = kind(theirs, **how)
    for p in theirs:
        p.grad = torch.ones_like(p)
    other.step()
    saved = other.state_dict()
    assert all("momentum_buffer" in s for s in saved["state"].values())
    opt = optim.Muon(parameters(), lr=0.25, momentum=0.5)
    before = opt.state_dict()
    with pytest.raises(ValueError, match=f"group 0 lacks .*{lacks}"):
        opt.load_state_dict(saved)
    assert opt.state_dict() == before and opt.param_groups[0]["lr"] == 0.25 and not opt.state


def test_its_own_checkpoint_is_loaded():
    opt, ps = optim.Muon(parameters(), lr=0.25, adjust=1.0), parameters()
    for p in opt.param_groups[0]["params"]:
        opt.state[p]["momentum_buffer"] = torch.full(p.shape, 2.0)
    other = optim.Muon(ps)
    for _ in range(2):
        other.load_state_dict(opt.state_dict())
    assert set(optim.Muon._OPTIONS) == set(opt.defaults)
    assert other.param_groups[0]["lr"] == 0.25 and other.param_groups[0]["adjust"] == 1.0
    assert all(torch.equal(other.state[p]["momentum_buffer"], torch.full(p.shape, 2.0)) for p in ps)


@pytest.mark.parametrize("bad,error", [(dict(adjust="none"), ValueError), (dict(adjust=None), TypeError),
                                       (dict(adjust=1.0, params=[torch.nn.Parameter(torch.ones(3))]), ValueError)],
                         ids=["name", "none", "vector"])
def test_a_refused_group_is_not_kept(bad, error):
    opt = optim.Muon(parameters())
    with pytest.raises(error):
        opt.add_param_group(dict(dict(params=parameters()), **bad))
    assert len(opt.param_groups) == 1
    opt.add_param_group(dict(params=parameters(), adjust="spectral"))
    assert len(opt.param_groups) == 2


def test_gradients_over_what_a_step_writes_are_refused(compiled):
    """Byte for byte: a gradient may lie right before or behind, and gradients over each other."""
    room = torch.ones(1000)
    cut = lambda at, rows=6, cols=8: room[at:at + rows * cols].view(rows, cols)
    plan = ops.MuonPlan([cut(100), cut(300)], [cut(148), cut(500)])
    for at in (0, 52, 196, 252, 348, 452, 548, 700):
        ops.dora_muon(plan, [cut(at), cut(at)], lr=0.1)
    for at, name in ((53, "params.0"), (100, "params.0"), (147, "params.0"), (148, "momenta.0"), (195, "momenta.0"),
                     (253, "params.1"), (347, "params.1"), (453, "momenta.1"), (547, "momenta.1")):
        steps = len(compiled.steps)
        for grads in ([cut(0), cut(at)], [cut(at), cut(0)]):
            with pytest.raises(ValueError, match=f"{name}. share memory"):
                ops.dora_muon(plan, grads, lr=0.1)
        assert len(compiled.steps) == steps
    p, w = torch.ones(6, 8, dtype=torch.bfloat16), torch.ones(6, 8)
    plan = ops.MuonPlan([p], [torch.zeros(6, 8)], masters=[w])
    with pytest.raises(ValueError, match="masters.0. share memory"):
        ops.dora_muon(plan, [w], lr=0.1)
    with pytest.raises(ValueError, match="params.0. share memory"):
        ops.dora_muon(plan, [p], lr=0.1)


@pytest.mark.parametrize("change", ["transposed", "type"])
@pytest.mark.parametrize("of", ["params", "momenta", "masters"])
def test_a_tensor_that_lies_otherwise_in_the_same_storage_is_refused(compiled, of, change):
    """Addresses and sizes are as they were; the step would take rows for columns, or bits for others."""
    p, m, w = torch.ones(8, 8, dtype=torch.bfloat16), torch.zeros(8, 8), torch.ones(8, 8)
    plan = ops.MuonPlan([p], [m], masters=[w])
    ops.dora_muon(plan, [torch.ones(8, 8)], lr=0.1)
    t = getattr(plan, of)[0]
    t.data = t.data.t() if change == "transposed" else t.data.view(torch.float16 if of == "params" else torch.int32)
    with pytest.raises(ValueError, match="contiguous|dtype|storage"):
        ops.dora_muon(plan, [torch.ones(8, 8)], lr=0.1)
    assert len(compiled.steps) == 1
