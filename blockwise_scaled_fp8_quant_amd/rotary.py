"""Rotary positions with autograd, and their frequencies, plain or scaled for contexts longer than those trained on.

The pages' model is built on the Qwen3-1.7B configuration, whose query and key heads are turned by their tokens' positions
between the qkv projection and the attention.  The turn is linear, its backward pass the turn back (puro_rotary, inverse).
"""
from __future__ import annotations

import math

import torch

from . import ROTARY_HALF, puro_rotary
from .linear import _apply

__all__ = ["Rotary", "RotaryFunction", "rotary", "rotary_frequencies"]


def rotary_frequencies(columns: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       trained_length: int | None = None, low: float = 1.0, high: float = 32.0, device=None):
    """(frequencies fp64 [columns / 2], radians a position; scale of the turned columns) for `columns` leading columns of a head:
    base^(-2 i / columns), and for contexts `factor` times as long as those trained on (trained_length positions)

      "linear"  positions divided by factor
      "base"    the base raised to base * factor^(columns / (columns - 2)): the slowest pair turns factor times slower, the
                fastest is left
      "yarn"    by turns over the trained length: pairs with fewer than `low` are slowed by factor, those with more than
                `high` left, those between mixed; scale 0.1 ln(factor) + 1 (Peng et al., "YaRN: Efficient Context Window
                Extension of Large Language Models", 2023, section 3)
    """
    if columns <= 0 or columns % 2:
        raise ValueError(f"columns {columns}: expected an even number above 0")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor: expected numbers above 0")
    if scaling == "base":
        if columns == 2:
            raise ValueError("one pair has no slower ones: 'base' needs 4 columns at least")
        base = base * factor ** (columns / (columns - 2))
    exponent = torch.arange(0, columns, 2, dtype=torch.float64, device=device) / columns
    freqs, scale = base ** -exponent, 1.0
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "yarn":
        if trained_length is None or not low < high:
            raise ValueError("'yarn' needs trained_length, and low < high")
        turns = trained_length * freqs / (2 * math.pi)
        kept = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        freqs = freqs / factor * (1 - kept) + freqs * kept
        scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f"scaling {scaling!r}: expected None, 'linear', 'base' or 'yarn'")
    return freqs, scale


class RotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, freqs, positions, start, layout, scale, inverse):
        ctx.save_for_backward(freqs, positions)
        ctx.how = (start, layout, scale, inverse)
        return puro_rotary(_heads(x), freqs, positions, start=start, layout=layout, scale=scale, inverse=inverse)

    @staticmethod
    def backward(ctx, dy):
        freqs, positions = ctx.saved_tensors
        start, layout, scale, inverse = ctx.how
        return RotaryFunction.apply(dy, freqs, positions, start, layout, scale, not inverse), None, None, None, None, None, None


def _heads(x):
    """x with unit stride in its heads (copied where it has none, such as a broadcast gradient)."""
    return x if x.stride(-1) == 1 or x.shape[-1] <= 1 else x.contiguous()


def rotary(x, freqs, positions=None, start: int = 0, layout: int = ROTARY_HALF, scale: float = 1.0):
    """x [tokens, heads, D] or [batch, tokens, heads, D], turned (differentiable).  positions: int64, of the leading dimensions
    of x or, the same for every sequence of a batch, [tokens]; None: start, start + 1, ... in every sequence."""
    if x.dim() not in (3, 4):
        raise ValueError(f"x: expected [tokens, heads, D] or [batch, tokens, heads, D], got shape {tuple(x.shape)}")
    lead = x.shape[:-2]
    if positions is not None and positions.shape not in (lead, lead[-1:]):
        raise ValueError(f"positions: shape {tuple(positions.shape)}, expected {tuple(lead)} or {tuple(lead[-1:])}")
    if x.dim() == 4:
        if positions is None:
            positions, start = torch.arange(start, start + lead[1], device=x.device), 0
        positions = positions.expand(lead).reshape(-1)
    flat = x if x.dim() == 3 else x.flatten(0, 1)
    if positions is not None:
        positions = positions.contiguous()
    return _apply(RotaryFunction, flat, freqs, positions, start, layout, scale, False).view(x.shape)


class Rotary(torch.nn.Module):
    """Rotary positions of the leading `columns` columns of every head; the arguments are those of rotary_frequencies."""

    def __init__(self, columns: int, base: float = 10000.0, layout: int = ROTARY_HALF, scaling: str | None = None, **how):
        super().__init__()
        self.columns, self.base, self.layout, self.scaling = columns, base, layout, scaling
        # no buffer: a module's cast to another type would round the frequencies
        with torch.inference_mode(False):
            self._freqs, self.scale = rotary_frequencies(columns, base, scaling, **how)
        self._copies = {self._freqs.device: self._freqs}

    def frequencies(self, device):
        """The frequencies on a device, copied there once.  The copy serves every later call, those with gradients too, whatever
        mode the first one is made in."""
        found = self._copies.get(device)
        if found is None:
            if device.type == "cuda" and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("a step is being captured before the frequencies are on its GPU: make the module there "
                                   "(device=), or one eager call first")
            with torch.inference_mode(False):
                # (from host memory, which the copy waits for: any stream may read it then)
                found = self._copies.setdefault(device, self._freqs.cpu().to(device))
        return found

    def forward(self, x, positions=None, start: int = 0):
        return rotary(x, self.frequencies(x.device), positions, start, self.layout, self.scale)

    def extra_repr(self) -> str:
        return f"{self.columns}, base={self.base}, scaling={self.scaling}"
