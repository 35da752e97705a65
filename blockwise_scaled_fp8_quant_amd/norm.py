"""Layer / RMS norm with autograd, alone and fused with the FP8 linear layer behind it.

The pages' model is built on the Qwen3-1.7B configuration: every block normalises its input and hands
it to FP8 linear layers (agihunt digest "清华用消费级 5090 花 6890 美元从零训 2B，15 项均分超过 Qwen2",
section 方法).  Fp8NormLinear is that pair, Y = norm(X) W^T for X [..., Din] (bf16 or fp32) and a bf16
W [Dout, Din]:

    forward   X -> 1x128 and 128x1 codes of norm(X), statistics   (puro_layer_norm_quant_dual)
              W -> 128x128 codes + transposed copy                (puro_fp8_quant_w_128x128)
              Y = FWD(codes, W)                                   bf16
    backward  dY -> 1x128 and 128x1 codes                         (puro_fp8_quant_act_dual)
              dN = DGRAD(dY, W^T copy)                            X's type
              dX, dweight, dbias = norm's backward(dN, X)         (puro_layer_norm_backward)
              dW = WGRAD(dY 128x1, norm(X) 128x1)                 fp32

norm(X) itself is never written.  Without gradients any number of rows is taken (single tokens, ragged
batches): puro_layer_norm_quant, then puro_gemm_rows.  fp32 `main_grad` tensors are added into as in
Fp8Linear.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (DGRAD, FWD, LAYER_NORM, OUT_BF16, OUT_FP32, RMS_NORM, WGRAD, puro_fp8_gemm, puro_fp8_gemm_accumulate,
               puro_fp8_quant_act_dual, puro_fp8_quant_w_128x128, puro_gemm_rows, puro_layer_norm,
               puro_layer_norm_backward, puro_layer_norm_quant, puro_layer_norm_quant_dual)
from .linear import Fp8Linear, _apply, _rows

__all__ = ["Norm", "NormFunction", "Fp8NormLinear", "Fp8NormLinearFunction", "layer_norm", "rms_norm"]


def _norm_grads(kind, dn, x2, gamma, mean, rstd, weight, bias, need_w, need_b):
    """dx and the weight's and bias's gradients of the norm (gamma: the weight as the forward pass saw it); those with
    a main_grad are added into it and returned as None."""
    main_w = getattr(weight, "main_grad", None) if need_w else None
    main_b = getattr(bias, "main_grad", None) if need_b else None
    if need_w and need_b and (main_w is None) != (main_b is None):
        raise ValueError("the norm's weight and bias need a main_grad both or neither")
    main = main_w is not None or main_b is not None
    if main:
        # the kernel adds into both; a parameter that needs no gradient gets a scratch tensor
        if main_w is None:
            main_w = torch.zeros(weight.shape, dtype=torch.float32, device=weight.device)
    dx, dw, db = puro_layer_norm_backward(dn, x2, gamma, mean, rstd, kind=kind, dweight=main_w, dbias=main_b,
                                          with_bias=need_b, accumulate=main)
    if main:
        return dx, None, None
    return dx, dw if need_w else None, db if need_b else None


class NormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, kind):
        x2 = _rows(x, x.shape[-1])
        y, mean, rstd = puro_layer_norm(x2, weight, bias, eps=eps, kind=kind)
        ctx.save_for_backward(x2, weight, mean, rstd)
        ctx.weight, ctx.bias, ctx.kind, ctx.x_shape = weight, bias, kind, x.shape
        return y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x2, gamma, mean, rstd = ctx.saved_tensors
        dx, dw, db = _norm_grads(ctx.kind, _rows(dy, x2.shape[1]), x2, gamma, mean, rstd, ctx.weight, ctx.bias,
                                 ctx.needs_input_grad[1], ctx.bias is not None and ctx.needs_input_grad[2])
        return dx.view(ctx.x_shape), dw, db, None, None


def layer_norm(x, weight, bias=None, eps: float = 1e-5):
    """Layer norm over the last dimension of x (differentiable)."""
    return _apply(NormFunction, x, weight, bias, eps, LAYER_NORM)


def rms_norm(x, weight, eps: float = 1e-6):
    """RMS norm over the last dimension of x (differentiable)."""
    return _apply(NormFunction, x, weight, None, eps, RMS_NORM)


class Norm(torch.nn.Module):
    """Layer norm (weight and bias) or RMS norm (weight), kind LAYER_NORM or RMS_NORM."""

    def __init__(self, features: int, kind: int = LAYER_NORM, eps: float = 1e-5, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.features, self.kind, self.eps = features, kind, eps
        self.weight = torch.nn.Parameter(torch.ones(features, dtype=dtype, device=device))
        self.bias = torch.nn.Parameter(torch.zeros(features, dtype=dtype, device=device)) if kind == LAYER_NORM else None

    def enable_main_grad(self):
        """Give the parameters fp32 gradient buffers that backward accumulates into."""
        for p in self.parameters():
            p.main_grad = torch.zeros(p.shape, dtype=torch.float32, device=p.device)

    def forward(self, x):
        return _apply(NormFunction, x, self.weight, self.bias, self.eps, self.kind)

    def extra_repr(self) -> str:
        return f"{self.features}, kind={'layer' if self.kind == LAYER_NORM else 'rms'}, eps={self.eps}"


class Fp8NormLinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, norm_weight, norm_bias, weight, eps, kind):
        dout, din = weight.shape
        x2 = _rows(x, din)
        xq, xs, xqT, xsT, mean, rstd = puro_layer_norm_quant_dual(x2, norm_weight, norm_bias, eps=eps, kind=kind)
        wq, ws, wqT, wsT = puro_fp8_quant_w_128x128(_rows(weight, din))
        y = puro_fp8_gemm(FWD, xq, xs, wq, ws, out_dtype=OUT_BF16)
        ctx.save_for_backward(x2, norm_weight, mean, rstd, xqT, xsT, wqT, wsT)
        ctx.params, ctx.kind, ctx.x_shape = (norm_weight, norm_bias, weight), kind, x.shape
        return y.view(*x.shape[:-1], dout)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x2, gamma, mean, rstd, xqT, xsT, wqT, wsT = ctx.saved_tensors
        norm_weight, norm_bias, weight = ctx.params
        if dy.dtype != torch.bfloat16:
            raise TypeError("Fp8NormLinear expects a bf16 output gradient")
        gq, gs, gqT, gsT = puro_fp8_quant_act_dual(_rows(dy, weight.shape[0]))
        need = ctx.needs_input_grad
        dx = dnw = dnb = dw = None
        if any(need[:3]):
            dn = puro_fp8_gemm(DGRAD, gq, gs, wqT, wsT, out_dtype=OUT_BF16 if x2.dtype == torch.bfloat16 else OUT_FP32)
            dx, dnw, dnb = _norm_grads(ctx.kind, dn, x2, gamma, mean, rstd, norm_weight, norm_bias, need[1],
                                       norm_bias is not None and need[2])
            dx = dx.view(ctx.x_shape)
        if need[3]:
            main = getattr(weight, "main_grad", None)
            if main is not None:
                puro_fp8_gemm_accumulate(WGRAD, gqT, gsT, xqT, xsT, main)
            else:
                dw = puro_fp8_gemm(WGRAD, gqT, gsT, xqT, xsT, out_dtype=OUT_FP32)
        return dx, dnw, dnb, dw, None, None


class Fp8NormLinear(torch.nn.Module):
    """Y = norm(X) W^T with the norm written straight as FP8 codes.  With gradients the number of rows must
    be a multiple of 128 (PuroError otherwise), as in Fp8Linear; without, any."""

    def __init__(self, in_features: int, out_features: int, kind: int = LAYER_NORM, eps: float = 1e-5, device=None):
        super().__init__()
        self.norm = Norm(in_features, kind, eps, device=device)
        self.linear = Fp8Linear(in_features, out_features, device=device)

    def enable_main_grad(self) -> None:
        self.norm.enable_main_grad()
        self.linear.enable_main_grad()

    def quantize_weight(self):
        """The linear weight's codes and scales, to be kept by a caller that runs many steps on one weight."""
        return self.linear.quantize_weight()

    def forward(self, x, codes=None):
        n, w = self.norm, self.linear.weight
        if x.shape[-1] != w.shape[1]:
            raise ValueError(f"x has {x.shape[-1]} features, weight expects {w.shape[1]}")
        if torch.is_grad_enabled():
            if codes is not None:
                raise ValueError("codes: a weight quantized beforehand is for use without gradients (torch.no_grad)")
            return _apply(Fp8NormLinearFunction, x, n.weight, n.bias, w, n.eps, n.kind)
        wq, ws = self.quantize_weight() if codes is None else codes
        xq, xs = puro_layer_norm_quant(_rows(x, w.shape[1]), n.weight, n.bias, eps=n.eps, kind=n.kind)
        return puro_gemm_rows(xq, xs, wq, ws).view(*x.shape[:-1], w.shape[0])
