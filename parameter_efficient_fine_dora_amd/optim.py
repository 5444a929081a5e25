"""AdamW for the adapters on top of the C ABI: every tensor of a parameter group in a few launches,
with moments in float32 or in 8-bit codes, float32 master weights and gradient clipping."""
from __future__ import annotations

import torch

from . import _lib, ops


class AdamW(torch.optim.Optimizer):
    """AdamW (decoupled weight decay) on contiguous bf16 or float32 device parameters.

    state_bits  32: float32 moments; 8: 8-bit codes with a scale per 128 elements (about 2 bytes a
                parameter for both moments instead of 8)
    master      keep a float32 copy of every bf16 parameter and update that; made from the parameter
                where a loaded state has none, and dropped from one where it is not wanted
    max_norm    clip the gradients of all groups together by their global norm; ``step`` then leaves
                the norm in ``grad_norm`` (a float32 scalar on the device).  Needs parameters of one
                dtype.

    Hyperparameters are read at each step, so schedulers work; they are kernel arguments, so a
    captured graph repeats the captured step's.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, *,
                 state_bits=32, master=False, max_norm=None):
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits is {state_bits}, expected 8 or 32")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay))
        self.state_bits, self.master, self.max_norm = state_bits, bool(master), max_norm
        self.grad_norm = None
        self._plans = {}

    def __getstate__(self):   # copies and pickles: torch's own parts, and the options
        return {**super().__getstate__(), "state_bits": self.state_bits, "master": self.master,
                "max_norm": self.max_norm}

    def __setstate__(self, state):
        super().__setstate__(state)
        self.grad_norm, self._plans = None, {}

    def _state_of(self, p):
        s = self.state[p]
        if not s:
            s["step"] = 0
            zero = torch.zeros_like(p, dtype=torch.float32, memory_format=torch.contiguous_format)
            if self.state_bits == 8:
                blocks = -(-p.numel() // _lib.STATE_BLOCK)
                s["exp_avg"] = torch.zeros_like(zero, dtype=torch.int8)
                s["exp_avg_sq"] = torch.zeros_like(zero, dtype=torch.uint8)
                s["exp_avg_scale"] = torch.zeros(blocks, dtype=torch.float32, device=p.device)
                s["exp_avg_sq_scale"] = torch.zeros(blocks, dtype=torch.float32, device=p.device)
            else:
                s["exp_avg"], s["exp_avg_sq"] = zero, torch.zeros_like(zero)
        if self._has_master(p):
            if "master" not in s:
                s["master"] = p.detach().float().contiguous()
        else:
            s.pop("master", None)
        return s

    def _has_master(self, p):
        return self.master and p.dtype == torch.bfloat16

    def _plan(self, slot, params):
        """The plan of these parameters, made anew when one of their tensors or its storage is
        another."""
        states = [self._state_of(p) for p in params]
        small = self.state_bits == 8
        lists = dict(exp_avg=[s["exp_avg"] for s in states], exp_avg_sq=[s["exp_avg_sq"] for s in states])
        if small:
            lists["exp_avg_scales"] = [s["exp_avg_scale"] for s in states]
            lists["exp_avg_sq_scales"] = [s["exp_avg_sq_scale"] for s in states]
        if self._has_master(params[0]):
            lists["masters"] = [s["master"] for s in states]
        kept = self._plans.get(slot)
        if kept is not None:
            plan, were = kept
            if (len(plan.params) == len(params) and all(a is b for a, b in zip(plan.params, params))
                    and all(a is b for k in lists for a, b in zip(lists[k], were[k]))
                    and plan.unchanged()):
                return plan
        plan = ops.AdamWPlan(params, lists["exp_avg"], lists["exp_avg_sq"], masters=lists.get("masters"),
                             exp_avg_scales=lists.get("exp_avg_scales"),
                             exp_avg_sq_scales=lists.get("exp_avg_sq_scales"))
        self._plans[slot] = (plan, lists)
        return plan

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        buckets = {}   # one call each: a group's parameters of one dtype, device and step count
        for gi, group in enumerate(self.param_groups):
            for p in group["params"]:
                if p.grad is not None:
                    key = (gi, p.dtype, p.grad.dtype, p.device, self._state_of(p)["step"])
                    buckets.setdefault(key, []).append(p)
        factor = None
        self.grad_norm = None
        if self.max_norm is not None and buckets:
            kinds = {k[1:4] for k in buckets}
            if len(kinds) != 1:
                raise ValueError("max_norm needs parameters of one dtype on one device")
            every = [p for ps in buckets.values() for p in ps]
            plan = self._plan("norm", every)
            self.grad_norm, factor = ops.dora_grad_norm(plan, [p.grad.contiguous() for p in every],
                                                        self.max_norm)
        used = {"norm"}
        for (gi, *rest, done), params in buckets.items():
            group = self.param_groups[gi]
            slot = (gi, *rest, params[0])   # step counts differ between buckets, first parameters too
            used.add(slot)
            ops.dora_adamw(self._plan(slot, params), [p.grad.contiguous() for p in params],
                           step=done + 1, lr=group["lr"], betas=group["betas"], eps=group["eps"],
                           weight_decay=group["weight_decay"], grad_scale=factor)
            for p in params:
                self.state[p]["step"] = done + 1
        self._plans = {k: v for k, v in self._plans.items() if k in used}
        return loss

    def _check_loadable(self, state_dict):
        """Refuses a checkpoint of an update that this one is not, and moments that it cannot use."""
        for group in state_dict["param_groups"]:
            for k in ("amsgrad", "maximize"):
                if group.get(k):
                    raise ValueError(f"a checkpoint with {k} is not supported")
            if not group.get("decoupled_weight_decay", True) and group.get("weight_decay"):
                raise ValueError("a checkpoint without decoupled weight decay is not supported")
        need = ["step", "exp_avg", "exp_avg_sq"]
        if self.state_bits == 8:
            need += ["exp_avg_scale", "exp_avg_sq_scale"]
        for i, s in state_dict["state"].items():
            if s and isinstance(s.get("exp_avg"), torch.Tensor):
                bits = 32 if s["exp_avg"].is_floating_point() else 8
                if bits != self.state_bits:
                    raise ValueError(f"the checkpoint has moments of {bits} bits, this optimizer "
                                     f"state_bits={self.state_bits}")
            lacks = [k for k in need if k not in s] if s else []
            if lacks:
                raise ValueError(f"the checkpoint's state of parameter {i} lacks {', '.join(lacks)}")

    def load_state_dict(self, state_dict):
        """Loads a checkpoint of this class, or of torch's AdamW (without amsgrad and maximize)."""
        self._check_loadable(state_dict)
        super().load_state_dict(state_dict)
        # torch casts floating state to the parameter's dtype; moments, codes and scales keep theirs
        # (all floating state here is float32), and step counts are numbers here
        ids = [i for g in state_dict["param_groups"] for i in g["params"]]
        mine = [p for g in self.param_groups for p in g["params"]]
        for i, p in zip(ids, mine):
            for k, v in state_dict["state"].get(i, {}).items():
                if k == "step":
                    v = int(v)
                elif isinstance(v, torch.Tensor):
                    v = v.detach().clone(memory_format=torch.contiguous_format).to(
                        p.device, torch.float32 if v.is_floating_point() else None)
                self.state[p][k] = v
        self._plans = {}
