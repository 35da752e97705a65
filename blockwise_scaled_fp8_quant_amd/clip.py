"""Clipping of a model's gradients by their global norm, for parameters whose gradients live in the fp32
`main_grad` buffers of the FP8 layers (Fp8Linear.enable_main_grad) or in `.grad`."""
from __future__ import annotations

from . import puro_clip_grad_norm, puro_grad_norm

__all__ = ["clip_grad_norm_", "gradients"]


def gradients(parameters):
    """The gradient tensors of parameters: main_grad where there is one, else .grad; each parameter once,
    those without a gradient left out."""
    if hasattr(parameters, "grad"):
        parameters = [parameters]
    found, seen = [], set()
    for p in parameters:
        if id(p) in seen:
            continue
        seen.add(id(p))
        g = getattr(p, "main_grad", None)
        g = p.grad if g is None else g
        if g is not None:
            found.append(g)
    return found


def clip_grad_norm_(parameters, max_norm: float):
    """Scale the gradients in place by min(1, max_norm / (norm + 1e-6)) and return their global norm (fp32, on the
    GPU; nothing waits for it).  A norm that is not finite reaches the gradients, as puro_ops.h says."""
    grads = gradients(parameters)
    if not grads:
        return puro_grad_norm(grads)
    return puro_clip_grad_norm(grads, max_norm)[0]
