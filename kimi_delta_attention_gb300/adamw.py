"""AdamW over the library's step for many tensors: a torch optimizer with states in 32 or 8 bits.

    opt = AdamW(layer.parameters(), lr=3e-3, state_bits=8)
    loss.backward(); opt.step(); opt.zero_grad()

All of a group's parameters go into one call (a launch for some 440 tensors).  States are fp32, or
e4m3 codes with a scale for 256 values, whatever the parameters' type.  In codes a second moment wanders about
its fp32 value by some 12 % at beta2 = 0.95, 20 % at 0.99 and 23 % at 0.999, and one below 1 / 229376 of the
largest of its 256 is held as that: such a value moves less than with fp32 states.  ``masters=True`` keeps an
fp32 copy of each bf16 parameter, of which the parameter is the rounded value.  With
``capturable=True`` the step numbers and the learning rate lie on the device, so that a captured
step goes on counting, and a schedule writes ``group["lr"].fill_(...)``.  Either way each parameter
counts the steps that it took; parameters whose counts differ go in calls of their own.  A step is
captured after at least one with the same gradients has been taken; others are refused.
"""
from __future__ import annotations

import torch

from ._adamw import BLOCK, E4M3, kda_adamw_step
from ._lib import KdaError


def _capturing():
    return torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()


def _before_capture(what):
    """Refuses to make what steps share during a capture: every replay would make it anew."""
    if _capturing():
        raise KdaError(1, f"a step under capture has no {what} yet: take one step with the same gradients before the capture")


def _on(device, t):
    """A word, or a number, on a device."""
    if torch.is_tensor(t) and t.device != device:
        _before_capture(f"word on {device} (one of its words lies on {t.device})")
        t = t.to(device)
    return t


class AdamW(torch.optim.Optimizer):
    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=32, masters=False, seed=0,
                 capturable=False):
        if state_bits not in (8, 32):
            raise KdaError(1, "state_bits must be 8 or 32")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay, state_bits=state_bits,
                                      masters=masters, seed=seed, capturable=capturable))

    def _init_state(self, p, group):
        st = self.state[p]
        st["step"] = 0
        for name in ("exp_avg", "exp_avg_sq"):
            if group["state_bits"] == 32:
                st[name] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
            else:
                st[name] = torch.zeros(p.numel(), dtype=torch.uint8, device=p.device).view(E4M3)
                st[name + "_scale"] = torch.zeros(-(-p.numel() // BLOCK), dtype=torch.float32, device=p.device)
        if group["masters"] and p.dtype != torch.float32:
            st["master"] = p.detach().float()

    def _device_words(self, group, params):
        """A capturable group's step numbers on the device: [(word, those of `params` that it counts for)].  Parameters
        that have taken the same number of steps share a word (the first one is the group's); a parameter
        without a gradient takes a word of its own along when the others go on."""
        joining, members, batches = {}, {}, {}
        for p in params:
            st = self.state[p]
            if "step_device" not in st:
                key = (p.device, st["step"])
                _before_capture("step number of a parameter on the device")
                if key not in joining:
                    joining[key] = torch.full((1,), st["step"], dtype=torch.int32, device=p.device)
                    group.setdefault("step_device", joining[key])
                st["step_device"] = joining[key]
            batches.setdefault(id(st["step_device"]), (st["step_device"], []))[1].append(p)
        for p in group["params"]:
            word = self.state[p].get("step_device") if p in self.state else None
            if word is not None:
                members.setdefault(id(word), []).append(p)
        for word, live in batches.values():
            if len(members[id(word)]) > len(live):
                _before_capture("step number apart for the parameters without a gradient")
                own, live = word.clone(), set(live)
                for p in members[id(word)]:
                    if p not in live:
                        self.state[p]["step_device"] = own
        return list(batches.values())

    def _device_lr(self, group, device):
        """The learning rate of a capturable group, on the device of its first parameter that steps."""
        if not torch.is_tensor(group["lr"]):
            _before_capture("learning rate on the device")
            group["lr"] = torch.full((1,), group["lr"], dtype=torch.float32, device=device)
        return group["lr"]

    @torch.no_grad()
    def step(self, closure=None, grad_scale=None, skip=None):
        """One step of every parameter that has a gradient; grad_scale and skip as kda_adamw_step's (a skipped
        step counts all the same).  A group's parameters may lie on several devices: words that lie on
        one of them are copied to the others."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            if not group["capturable"] and _capturing():
                raise KdaError(1, "a step under capture needs capturable=True: every replay would take the same step number")
            live = [p for p in group["params"] if p.grad is not None]
            for p in live:
                if p.grad.is_sparse:
                    raise KdaError(1, "sparse gradients are not supported")
                if not self.state[p]:
                    _before_capture("state of a parameter")
                    self._init_state(p, group)
            if group["capturable"]:
                batches = self._device_words(group, live)
            else:
                group.pop("step_device", None)
                alike = {}                  # parameters that have taken the same number of steps, device by device
                for p in live:
                    st = self.state[p]
                    if "step_device" in st:  # (it was capturable: replays have counted there alone)
                        st["step"] = int(st.pop("step_device"))
                    alike.setdefault((p.device, st["step"] + 1), []).append(p)
                batches = [(step, params) for (_, step), params in alike.items()]
            for step, params in batches:
                device, lr = params[0].device, group["lr"]
                if group["capturable"]:
                    lr = self._device_lr(group, device)
                    step.add_(1)
                states = [self.state[p] for p in params]
                column = lambda name: [s[name] for s in states]
                here = lambda t: _on(device, t)
                small = group["state_bits"] == 8
                try:
                    kda_adamw_step(params, [p.grad.contiguous() for p in params], column("exp_avg"), column("exp_avg_sq"), step,
                                   lr=here(lr), betas=group["betas"], eps=group["eps"], weight_decay=group["weight_decay"],
                                   masters=[s.get("master") for s in states] if group["masters"] else None,
                                   exp_avg_scales=column("exp_avg_scale") if small else None,
                                   exp_avg_sq_scales=column("exp_avg_sq_scale") if small else None, seed=group["seed"],
                                   grad_scale=here(grad_scale), skip=here(skip))
                except Exception:           # (a call that was refused has not counted)
                    if group["capturable"]:
                        step.sub_(1)
                    raise
                for st in states:
                    st["step"] += 1
        return loss

    def load_state_dict(self, state_dict):
        super().load_state_dict(state_dict)
        for group, saved in zip(self.param_groups, state_dict["param_groups"]):
            # (torch casts floating states to their parameter's type: put them back as they were)
            params = [(p, state_dict["state"][i]) for i, p in zip(saved["params"], group["params"]) if i in state_dict["state"]]
            for p, state in params:
                for name, value in state.items():
                    if torch.is_tensor(value) and name != "step_device":
                        self.state[p][name] = value.detach().clone().to(p.device)
            if not params:
                continue
            device = params[0][0].device
            if torch.is_tensor(group["lr"]):
                group["lr"] = group["lr"].to(device)
            if not group["capturable"]:
                continue
            # counts alike share a word again (a state without one, of an older file, has the group's)
            counts = {id(t): int(t) for t in [saved.get("step_device")] + [s.get("step_device") for _, s in params] if t is not None}
            words = {}
            word = lambda d, n: words.setdefault((d, n), torch.full((1,), n, dtype=torch.int32, device=d))
            for p, state in params:
                t = state.get("step_device", saved.get("step_device"))
                self.state[p]["step_device"] = word(p.device, state["step"] if t is None else counts[id(t)])
            if saved.get("step_device") is not None:
                group["step_device"] = word(device, counts[id(saved["step_device"])])
