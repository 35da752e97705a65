"""AdamW over all parameters of a model at once, for gradients in the fp32 `main_grad` buffers of the FP8 layers
(Fp8Linear.enable_main_grad) or in `.grad`.

The method keeps master weights and optimizer state in BF16/FP32 (agihunt digest "清华用消费级 5090 花 6890 美元从零训 2B，
15 项均分超过 Qwen2", section 方法, FP8 bullet) and trains what is no matrix with AdamW.  bf16 parameters get an fp32 master copy
here, states are fp32 or, at a quarter of the memory, 8-bit (include/puro_ops.h: puro_adamw); clipping by the global
norm costs no pass over the gradients of its own.
"""
from __future__ import annotations

import torch

from . import puro_adamw, puro_grad_norm
from .clip import gradients

__all__ = ["AdamW"]

_STATES = ("exp_avg", "exp_avg_sq", "avg_scale", "sq_scale", "master")


class AdamW(torch.optim.Optimizer):
    """Options, of all groups or of each: lr (a number, or an fp32 tensor of one value on the GPU), betas, eps, weight_decay;
    state_bits: 32, or 8.  master_weights: keep an fp32 copy of each bf16 parameter, of which the parameter is the
    rounding (without one, a step smaller than half the distance of two bf16 numbers is lost).  seed: of the rounding of
    8-bit states.  capturable: the count of steps lives on the GPU, so that a step may be captured into a graph; every
    parameter of the group then has a gradient at every step."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 state_bits: int = 32, master_weights: bool = True, seed: int = 0, capturable: bool = False):
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay, state_bits=state_bits,
                                      master_weights=master_weights, seed=seed, capturable=capturable))

    def add_param_group(self, group):
        super().add_param_group(group)
        if self.param_groups[-1]["state_bits"] not in (8, 32):
            raise ValueError(f"state_bits {self.param_groups.pop()['state_bits']}: expected 8 or 32")

    def _init(self, p, group):
        """The state of a parameter without one."""
        if p.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"parameters are bf16 or fp32, not {p.dtype}")
        s = self.state[p]
        codes = group["state_bits"] == 8
        for name in _STATES[:2]:
            s[name] = torch.zeros_like(p, dtype=torch.uint8 if codes else torch.float32)
        for name in _STATES[2:4] if codes else ():
            s[name] = torch.zeros((p.numel() + 127) // 128, dtype=torch.float32, device=p.device)
        if p.dtype == torch.bfloat16 and group["master_weights"]:
            s["master"] = p.detach().float()
        s["step"] = torch.zeros((), dtype=torch.int64, device=p.device) if group["capturable"] else 0
        return s

    def sync_masters(self):
        """Take the master copies from the parameters again: after something else has changed those."""
        with torch.no_grad():
            for p, s in self.state.items():
                if "master" in s:
                    s["master"].copy_(p)

    def zero_grad(self, set_to_none: bool = True):
        """As torch's; main_grad buffers are set to zero and stay."""
        super().zero_grad(set_to_none)
        for group in self.param_groups:
            for p in group["params"]:
                main = getattr(p, "main_grad", None)
                if main is not None:
                    main.zero_()

    @torch.no_grad()
    def step(self, closure=None, *, max_norm: float | None = None):
        """One step.  max_norm: the gradients are taken times min(1, max_norm / (norm + 1e-6)), with the norm of all of
        them, which is then in grad_norm (fp32, on the GPU; nothing waits for it); they themselves stay as they are."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        norm = None
        if max_norm is not None:
            norm = self.grad_norm = puro_grad_norm(gradients([p for g in self.param_groups for p in g["params"]]))
        for k, group in enumerate(self.param_groups):
            members = self._capturable(group) if group["capturable"] else self._counted(group)
            for step, params, grads in members:
                states = [self.state[p] for p in params]

                def column(name):
                    return [s.get(name) for s in states] if any(name in s for s in states) else None
                if group["capturable"]:
                    step.add_(1)
                try:
                    puro_adamw(params, grads, column("exp_avg"), column("exp_avg_sq"), step, group["lr"], *group["betas"],
                               group["eps"], group["weight_decay"], masters=column("master"), avg_scales=column("avg_scale"),
                               sq_scales=column("sq_scale"), norm=norm, max_norm=1.0 if norm is None else max_norm,
                               seed=(group["seed"] + k * 0x9E3779B97F4A7C15) % 2 ** 64)
                except Exception:
                    if group["capturable"]:
                        step.sub_(1)                  # a refused step is none
                    raise
                if not group["capturable"]:
                    for s in states:
                        s["step"] = step
        return loss

    def _gradient(self, p):
        """The parameter's gradient in its layout, or None."""
        found = gradients(p)
        if not found:
            return None
        g = found[0]
        if g.layout != torch.strided:
            raise TypeError("sparse gradients are not supported")
        if g.stride() != p.stride() and not (g.is_contiguous() and p.is_contiguous()):
            g = torch.empty_like(p, dtype=g.dtype).copy_(g)            # (as a broadcast gradient)
        return g

    def _counted(self, group):
        """[(number of the step, parameters, gradients)] of those with a gradient, by how many steps they have had."""
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a step is being captured: AdamW(capturable=True) counts its steps on the GPU")
        by_step = {}
        for p in group["params"]:
            g = self._gradient(p)
            if g is None:
                continue
            step = (self.state[p] or self._init(p, group))["step"] + 1
            _, params, grads = by_step.setdefault(step, (step, [], []))
            params.append(p)
            grads.append(g)
        return list(by_step.values())

    def _capturable(self, group):
        """[(the count, parameters, gradients)]: one count, on the GPU, for the whole group."""
        params = list(group["params"])
        grads = [self._gradient(p) for p in params]
        if any(g is None for g in grads):
            raise RuntimeError("a capturable AdamW needs a gradient of every parameter at every step")
        capturing = torch.cuda.is_current_stream_capturing()
        if capturing and not all(self.state[p] for p in params):
            raise RuntimeError("a step is being captured before the first eager one: every replay would make the states anew")
        states = [self.state[p] or self._init(p, group) for p in params]
        if not states:
            return []
        count = states[0]["step"]
        if any(s["step"] is not count for s in states):
            if capturing:
                raise RuntimeError("a step is being captured before the first eager one")
            if any(int(s["step"]) != int(count) for s in states):
                raise RuntimeError("the parameters of a capturable group have to have had the same number of steps")
            for s in states:
                s["step"] = count
        return [(count, params, grads)]

    def load_state_dict(self, state_dict):
        """As torch's, but for the states' types: torch casts them to the parameters'."""
        super().load_state_dict(state_dict)
        saved = [i for group in state_dict["param_groups"] for i in group["params"]]
        mine = [(p, group) for group in self.param_groups for p in group["params"]]
        for i, (p, group) in zip(saved, mine):
            if i not in state_dict["state"]:
                continue
            given, s = state_dict["state"][i], self.state[p]
            for name in _STATES:
                if name in given:
                    s[name] = given[name].detach().to(p.device, copy=True)
            count = int(given["step"])
            s["step"] = torch.full((), count, dtype=torch.int64, device=p.device) if group["capturable"] else count
