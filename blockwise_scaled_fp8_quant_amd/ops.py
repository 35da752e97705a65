"""Python binding of the operators around the FP8 linear layer (``include/puro_ops.h``): the norm in
front of it, forward (as a tensor, as 1x128 codes, as 1x128 and transposed 128x1 codes) and backward,
the product of those codes for any number of rows, and the clipping of gradients by their global norm.

Argument marshalling only, by the rules of the package: tensors on the current GPU, outputs and
workspaces allocated where not given, TypeError or ValueError for what the C ABI cannot see, PuroError
for a non-zero status, nothing launched in either case.  (A dimension of one element may carry any stride,
as in is_contiguous, and rows may be any distance apart that is no less than their length.)  The marshalling
itself is native (csrc/marshal.cpp): a decode step makes these calls by the thousand.

Every function takes `stream`, a torch stream or a handle as in `cuda_stream` (0 is the default stream's): the call
then runs as under torch.cuda.stream, so what it allocates (outputs, workspace) comes from that stream's memory and is
not handed out again before the work on it is done.  A caller that uses such an output on another stream orders the
two, as for any tensor.

The functions are available from the package.
"""
from __future__ import annotations

import ctypes

import torch

from . import OUT_BF16, PuroError, _i64, _int, _p, _sz, lib


class _Unavailable:
    """In the place of the marshalling where it is not built or does not load: the entry points of puro_fp8.h work
    without it, those here say what is missing."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"_marshal.so beside ops.py is needed for this call ({self._why}): build it (python "
                          "blockwise_scaled_fp8_quant_amd/build.py or __graft_entry__.build())")


try:
    from . import _marshal
except ImportError as _error:
    _marshal = _Unavailable(_error)

__all__ = [
    "LAYER_NORM", "RMS_NORM", "EXPORTED_OPS", "GradJob", "puro_layer_norm", "puro_layer_norm_quant",
    "puro_layer_norm_quant_dual", "puro_layer_norm_backward", "puro_layer_norm_backward_workspace_size",
    "puro_grad_norm", "puro_clip_grad_norm", "puro_scale_by_norm", "puro_gemm_rows", "puro_gemm_rows_workspace_size",
]

LAYER_NORM, RMS_NORM = 0, 1

EXPORTED_OPS = (
    "puro_layer_norm", "puro_layer_norm_quant", "puro_layer_norm_quant_dual", "puro_layer_norm_backward",
    "puro_layer_norm_backward_workspace_size", "puro_grad_norm", "puro_clip_grad_norm", "puro_scale_by_norm",
    "puro_grad_norm_workspace_size", "puro_gemm_rows", "puro_gemm_rows_workspace_size",
)

_f32 = ctypes.c_float


class GradJob(ctypes.Structure):
    """puro_grad_job (include/puro_ops.h): one gradient tensor, and where its clipped values go."""
    _fields_ = [("src", _p), ("dst", _p), ("n", _i64), ("dtype", _int)]


_norm_in = [_int, _int, _p, _i64, _i64, _i64, _int, _p, _p, _f32]
lib.puro_layer_norm.argtypes = _norm_in + [_p, _i64, _p, _p, _p]
lib.puro_layer_norm_quant.argtypes = _norm_in + [_p, _i64, _p, _p, _p, _p]
lib.puro_layer_norm_quant_dual.argtypes = _norm_in + [_p, _i64, _p, _p, _i64, _p, _p, _p, _p]
lib.puro_layer_norm_backward.argtypes = [_int, _int, _p, _i64, _p, _i64, _i64, _i64, _int, _p, _p, _p, _p, _i64, _p, _p,
                                         _int, _p, _sz, _p]
lib.puro_layer_norm_backward_workspace_size.argtypes = [_i64, _i64]
lib.puro_grad_norm.argtypes = [_p, _int, _p, _p, _sz, _p]
lib.puro_clip_grad_norm.argtypes = [_p, _int, _f32, _p, _p, _sz, _p]
lib.puro_scale_by_norm.argtypes = [_p, _int, _f32, _p, _p]
lib.puro_grad_norm_workspace_size.argtypes = [_p, _int]
lib.puro_gemm_rows.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _p, _i64, _p, _p, _i64, _int, _p, _sz, _p]
lib.puro_gemm_rows_workspace_size.argtypes = [_i64, _i64, _i64]
for _f in EXPORTED_OPS:
    getattr(lib, _f).restype = _sz if _f.endswith("_workspace_size") else _int


def _device() -> int:
    """The current GPU's index; one that no tensor has where there is no GPU (every check then refuses)."""
    try:
        return torch._C._cuda_getDevice()
    except RuntimeError:
        return -2


def _raise(status: int, where: str):
    raise PuroError(status, where)


if not isinstance(_marshal, _Unavailable):
    _marshal.init(_device, torch._C._cuda_getCurrentRawStream, _raise)


def check_capture(tensors):
    """Refuse (RuntimeError) a step that is being captured over the living autograd graph of another stream, which would
    end the process; tensors: the inputs and parameters of a differentiable call."""
    _marshal.check_capture(tensors)


def _on(stream, call):
    """`call`, on the stream named (a torch stream or a raw handle; ExternalStream takes the handle 0, the default
    stream's, for none given, and makes a stream that nothing orders)."""
    if stream is None:
        return call
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()

    def run(*args):
        with torch.cuda.stream(stream):
            return call(*args)
    return run


def puro_layer_norm(x, weight, bias=None, eps: float = 1e-5, kind: int = LAYER_NORM, y=None, mean=None, rstd=None,
                    stats: bool = True, stream=None):
    """x [T, C] bf16 or fp32 -> (y [T, C] of x's type, mean fp32 [T], rstd fp32 [T]): the layer or RMS norm
    of each row and the statistics its backward pass takes.  mean is None for RMS_NORM; with stats=False
    only the statistics given are written; those of rows without columns are NaN.  y may be x."""
    return _on(stream, _marshal.layer_norm)(x, weight, bias, eps, kind, y, mean, rstd, stats)


def puro_layer_norm_quant(x, weight, bias=None, eps: float = 1e-5, kind: int = LAYER_NORM, q=None, s=None, mean=None,
                          rstd=None, stream=None):
    """x [T, C] -> (q uint8 [T, C], s fp32 [C/128, T]): the norm of each row as 1x128 codes and scales
    (layouts of puro_fp8_quant_act_1x128), for any T.  mean and rstd are written where given."""
    return _on(stream, _marshal.layer_norm_quant)(x, weight, bias, eps, kind, q, s, mean, rstd)


def puro_layer_norm_quant_dual(x, weight, bias=None, eps: float = 1e-5, kind: int = LAYER_NORM, q=None, s=None, qT=None,
                               sT=None, mean=None, rstd=None, stream=None):
    """x [T, C] -> (q [T, C], s [C/128, T], qT [C, T], sT [T/128, C], mean, rstd): the norm of each row as the
    codes and scales of both orientations (layouts of puro_fp8_quant_act_dual), and its statistics."""
    return _on(stream, _marshal.layer_norm_quant_dual)(x, weight, bias, eps, kind, q, s, qT, sT, mean, rstd)


def puro_layer_norm_backward_workspace_size(T: int, C: int) -> int:
    return lib.puro_layer_norm_backward_workspace_size(T, C)


def puro_layer_norm_backward(dy, x, weight, mean, rstd, kind: int = LAYER_NORM, dx=None, dweight=None, dbias=None,
                             with_bias: bool = True, accumulate: bool = False, workspace=None, stream=None):
    """(dx [T, C] of x's type, dweight fp32 [C], dbias fp32 [C] or None): the backward pass of the norm, from
    the statistics of the forward pass (mean is None for RMS_NORM).  accumulate adds to the dweight and dbias given.
    dx may be dy or x."""
    return _on(stream, _marshal.layer_norm_backward)(dy, x, weight, mean, rstd, kind, dx, dweight, dbias, with_bias,
                                                     accumulate, workspace)


def puro_grad_norm(grads, norm=None, workspace=None, stream=None):
    """norm (fp32, one value, on the GPU): the square root of the sum of all squares of a list of bf16 or fp32
    tensors, each contiguous or dense in another order of its dimensions."""
    return _on(stream, _marshal.clip_grad_norm)(list(grads), None, None, norm, workspace)


def puro_clip_grad_norm(grads, max_norm: float, outs=None, norm=None, workspace=None, stream=None):
    """(norm, outs): the global norm of a list of tensors as puro_grad_norm takes them, and the tensors times
    min(1, max_norm / (norm + 1e-6)) -- in place (outs is then grads), or into the tensors given as outs, of the same
    types, shapes and layouts."""
    grads = list(grads)
    if max_norm is None:
        raise TypeError("max_norm: expected a number")
    norm = _on(stream, _marshal.clip_grad_norm)(grads, max_norm, None if outs is None else list(outs), norm, workspace)
    return norm, grads if outs is None else outs


def puro_scale_by_norm(grads, max_norm: float, norm, outs=None, stream=None):
    """The tensors times min(1, max_norm / (norm + 1e-6)) with a norm already on the GPU (for instance joined
    over processes); in place, or into outs.  Returns the tensors written."""
    grads = list(grads)
    _on(stream, _marshal.scale_by_norm)(grads, max_norm, norm, None if outs is None else list(outs))
    return grads if outs is None else outs


def puro_gemm_rows_workspace_size(M: int, N: int, K: int) -> int:
    return lib.puro_gemm_rows_workspace_size(M, N, K)


def puro_gemm_rows(A, sA, B, sB, C=None, out_dtype: int = OUT_BF16, workspace=None, stream=None):
    """C [M, N] = blockwise-scaled FP8 product of A [M, K] (sA fp32 [K/128, M]) and B [N, K] (sB fp32
    [N/128, K/128]) for any number of rows M; see puro_ops.h."""
    return _on(stream, _marshal.gemm_rows)(A, sA, B, sB, C, out_dtype, workspace)
