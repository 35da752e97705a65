"""The residual sum behind a block together with the norm in front of the next one, with autograd, alone and fused with the
FP8 linear layer that reads the norm.

    h_out = h + scale * gate * p,   p = x or norm(x) * post_weight;   y = norm(h_out) * weight + bias

The pages' model is built on the Qwen3-1.7B configuration (agihunt digest "清华用消费级 5090 花 6890 美元从零训 2B，15 项均分
超过 Qwen2", section 方法), whose blocks add their output to the residual stream and normalise it again in front of the next
FP8 linear layers; there gate and post_weight are absent and scale is 1.  Fp8ResidualNormLinear is that sequence,
(h, x) -> (norm(h + x) W^T, h + x):

    forward   h, x -> h_out, 1x128 and 128x1 codes of the norm, statistics  (puro_residual_norm_quant_dual)
              W -> 128x128 codes + transposed copy                          (puro_fp8_quant_w_128x128)
              Y = FWD(codes, W)                                             bf16
    backward  dY -> codes of both orientations, dN = DGRAD, dW = WGRAD      as Fp8NormLinear
              dh, dx, the vectors' gradients = backward(dN, dh_out)         (puro_residual_norm_backward)

The norm itself is never written.  Without gradients any number of rows is taken.  fp32 `main_grad` tensors are added into as
in Fp8Linear.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (DGRAD, FWD, LAYER_NORM, OUT_BF16, OUT_FP32, WGRAD, puro_fp8_gemm, puro_fp8_gemm_accumulate,
               puro_fp8_quant_act_dual, puro_fp8_quant_w_128x128, puro_gemm_rows, puro_residual_norm,
               puro_residual_norm_backward, puro_residual_norm_quant, puro_residual_norm_quant_dual)
from .linear import Fp8Linear, _apply, _rows

__all__ = ["ResidualNorm", "ResidualNormFunction", "Fp8ResidualNormLinear", "Fp8ResidualNormLinearFunction", "residual_norm"]


def _residual_grads(ctx, dn, dh_out, saved, needs):
    """(dh, dx, dweight, dbias, dgate, dpost_weight) from the gradients of the norm and of the sum (None for zero), as
    autograd takes them; saved: (h_out, x, weight, gate, post_weight, mean, rstd, post_mean, post_rstd) as the forward pass saw
    them; needs: of h, x and the four vectors.  Vectors with a main_grad are added into it and returned as None."""
    h_out, x, weight, gate, post, mean, rstd, post_mean, post_rstd = saved
    C = h_out.shape[1]
    vectors = dict(zip(("dweight", "dbias", "dgate", "dpost_weight"), ctx.vectors))      # the parameters themselves
    wanted = [k for (k, v), need in zip(vectors.items(), needs[2:]) if v is not None and need]
    mains = {k: getattr(vectors[k], "main_grad", None) for k in wanted}
    main = any(v is not None for v in mains.values())
    if main and any(v is None for v in mains.values()):
        raise ValueError("the vectors of a residual sum and norm need a main_grad all or none")
    into = {}
    if main:
        # the kernel adds into all of them; a parameter that needs no gradient gets a scratch tensor
        into = {k: mains.get(k) if k in mains else torch.zeros(C, dtype=torch.float32, device=h_out.device)
                for k, v in vectors.items() if v is not None and (k != "dbias" or "dbias" in wanted)}
    dn = torch.zeros_like(h_out) if dn is None else _rows(dn, C)
    dh_out = None if dh_out is None else _rows(dh_out, C)
    out = puro_residual_norm_backward(dn, h_out, weight, mean, rstd, x=x, gate=gate, post_weight=post, post_mean=post_mean,
                                      post_rstd=post_rstd, dh_out=dh_out, scale=ctx.scale, kind=ctx.kind,
                                      with_bias="dbias" in wanted, accumulate=main, **into)
    dh = out[0].view(ctx.shape)
    # (where both are one tensor autograd has to see that they are, or two leaves would take the same memory for theirs)
    dx = dh if out[1] is out[0] else out[1].view(ctx.shape)
    return [dh, dx] + [g if not main and k in wanted else None for k, g in zip(vectors, out[2:])]


class ResidualNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, x, weight, bias, gate, post_weight, eps, kind, scale):
        if x.shape != h.shape:
            raise ValueError(f"x has shape {tuple(x.shape)}, the residual stream {tuple(h.shape)}")
        C = h.shape[-1]
        x2 = _rows(x, C)
        y, h_out, *stats = puro_residual_norm(_rows(h, C), x2, weight, bias, eps=eps, kind=kind, gate=gate,
                                              post_weight=post_weight, scale=scale)
        gated = gate is not None or post_weight is not None
        ctx.save_for_backward(h_out, x2 if gated else None, weight, gate, post_weight, *stats)
        ctx.vectors, ctx.kind, ctx.scale, ctx.shape = (weight, bias, gate, post_weight), kind, scale, h.shape
        ctx.set_materialize_grads(False)
        return y.view(h.shape), h_out.view(h.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_out):
        grads = _residual_grads(ctx, dy, dh_out, ctx.saved_tensors, ctx.needs_input_grad[:6])
        return *grads, None, None, None


def residual_norm(h, x, weight, bias=None, gate=None, post_weight=None, eps: float = 1e-5, kind: int = LAYER_NORM,
                  scale: float = 1.0):
    """(y, h_out) over the last dimension of the residual stream h and a block's output x (differentiable)."""
    return _apply(ResidualNormFunction, h, x, weight, bias, gate, post_weight, eps, kind, scale)


class ResidualNorm(torch.nn.Module):
    """(h, x) -> (y, h_out).  kind LAYER_NORM (weight and bias) or RMS_NORM (weight).  gate: a factor per channel that starts
    at this value (None: none); post_norm: a norm of the block's output, with a weight; scale: a constant factor."""

    def __init__(self, features: int, kind: int = LAYER_NORM, eps: float = 1e-5, gate: float | None = None,
                 post_norm: bool = False, scale: float = 1.0, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.features, self.kind, self.eps, self.scale = features, kind, eps, scale

        def vector(value):
            return torch.nn.Parameter(torch.full((features,), value, dtype=dtype, device=device))
        self.weight = vector(1.0)
        self.bias = vector(0.0) if kind == LAYER_NORM else None
        self.gate = None if gate is None else vector(gate)
        self.post_weight = vector(1.0) if post_norm else None

    def enable_main_grad(self):
        """Give the parameters fp32 gradient buffers that backward accumulates into."""
        for p in self.parameters():
            p.main_grad = torch.zeros(p.shape, dtype=torch.float32, device=p.device)

    def forward(self, h, x):
        return _apply(ResidualNormFunction, h, x, self.weight, self.bias, self.gate, self.post_weight, self.eps, self.kind,
                      self.scale)

    def extra_repr(self) -> str:
        return (f"{self.features}, kind={'layer' if self.kind == LAYER_NORM else 'rms'}, eps={self.eps}, scale={self.scale}, "
                f"gate={self.gate is not None}, post_norm={self.post_weight is not None}")


class Fp8ResidualNormLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, x, norm_weight, norm_bias, gate, post_weight, weight, eps, kind, scale):
        if x.shape != h.shape:
            raise ValueError(f"x has shape {tuple(x.shape)}, the residual stream {tuple(h.shape)}")
        dout, din = weight.shape
        x2 = _rows(x, din)
        q, s, qT, sT, h_out, *stats = puro_residual_norm_quant_dual(_rows(h, din), x2, norm_weight, norm_bias, eps=eps, kind=kind,
                                                                    gate=gate, post_weight=post_weight, scale=scale)
        wq, ws, wqT, wsT = puro_fp8_quant_w_128x128(_rows(weight, din))
        y = puro_fp8_gemm(FWD, q, s, wq, ws, out_dtype=OUT_BF16)
        gated = gate is not None or post_weight is not None
        ctx.save_for_backward(h_out, x2 if gated else None, norm_weight, gate, post_weight, *stats, qT, sT, wqT, wsT)
        ctx.vectors, ctx.weight = (norm_weight, norm_bias, gate, post_weight), weight
        ctx.kind, ctx.scale, ctx.shape = kind, scale, h.shape
        ctx.set_materialize_grads(False)
        return y.view(*h.shape[:-1], dout), h_out.view(h.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_out):
        *saved, qT, sT, wqT, wsT = ctx.saved_tensors
        need, weight = ctx.needs_input_grad, ctx.weight
        dn = dw = None
        if dy is not None:
            if dy.dtype != torch.bfloat16:
                raise TypeError("Fp8ResidualNormLinear expects a bf16 output gradient")
            gq, gs, gqT, gsT = puro_fp8_quant_act_dual(_rows(dy, weight.shape[0]))
            if any(need[:6]):
                dn = puro_fp8_gemm(DGRAD, gq, gs, wqT, wsT, out_dtype=OUT_BF16 if saved[0].dtype == torch.bfloat16 else OUT_FP32)
            if need[6]:
                main = getattr(weight, "main_grad", None)
                if main is not None:
                    puro_fp8_gemm_accumulate(WGRAD, gqT, gsT, qT, sT, main)
                else:
                    dw = puro_fp8_gemm(WGRAD, gqT, gsT, qT, sT, out_dtype=OUT_FP32)
        grads = _residual_grads(ctx, dn, dh_out, saved, need[:6]) if any(need[:6]) else [None] * 6
        return *grads, dw, None, None, None


class Fp8ResidualNormLinear(torch.nn.Module):
    """(h, x) -> (norm(h_out) W^T, h_out) with h_out the residual sum, the norm written straight as FP8 codes.  With gradients
    the number of rows must be a multiple of 128 (PuroError otherwise), as in Fp8Linear; without, any.  gate, post_norm
    and scale as in ResidualNorm."""

    def __init__(self, in_features: int, out_features: int, kind: int = LAYER_NORM, eps: float = 1e-5,
                 gate: float | None = None, post_norm: bool = False, scale: float = 1.0, device=None):
        super().__init__()
        self.norm = ResidualNorm(in_features, kind, eps, gate, post_norm, scale, device=device)
        self.linear = Fp8Linear(in_features, out_features, device=device)

    def enable_main_grad(self) -> None:
        self.norm.enable_main_grad()
        self.linear.enable_main_grad()

    def quantize_weight(self):
        """The linear weight's codes and scales, to be kept by a caller that runs many steps on one weight."""
        return self.linear.quantize_weight()

    def forward(self, h, x, codes=None):
        n, w = self.norm, self.linear.weight
        if h.shape[-1] != w.shape[1]:
            raise ValueError(f"h has {h.shape[-1]} features, weight expects {w.shape[1]}")
        if torch.is_grad_enabled():
            if codes is not None:
                raise ValueError("codes: a weight quantized beforehand is for use without gradients (torch.no_grad)")
            return _apply(Fp8ResidualNormLinearFunction, h, x, n.weight, n.bias, n.gate, n.post_weight, w, n.eps, n.kind, n.scale)
        if x.shape != h.shape:
            raise ValueError(f"x has shape {tuple(x.shape)}, the residual stream {tuple(h.shape)}")
        wq, ws = self.quantize_weight() if codes is None else codes
        q, s, h_out = puro_residual_norm_quant(_rows(h, w.shape[1]), _rows(x, w.shape[1]), n.weight, n.bias, eps=n.eps, kind=n.kind,
                                               gate=n.gate, post_weight=n.post_weight, scale=n.scale)
        return puro_gemm_rows(q, s, wq, ws).view(*h.shape[:-1], w.shape[0]), h_out.view(h.shape)
