"""Python binding of the operators around the FP8 linear layer (``include/puro_ops.h``): the norm in
front of it, forward (as a tensor, as 1x128 codes, as 1x128 and transposed 128x1 codes) and backward,
the product of those codes for any number of rows, and the clipping of gradients by their global norm.

Argument marshalling only, by the rules of the package: tensors on the current GPU, outputs and
workspaces allocated where not given, TypeError or ValueError for what the C ABI cannot see, PuroError
for a non-zero status, nothing launched in either case.  The functions are available from the package.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import OUT_BF16, OUT_FP32, PuroError, _check, _i64, _int, _need, _p, _stream, _sz, lib

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


_jobs = ctypes.POINTER(GradJob)
_norm_in = [_int, _int, _p, _i64, _i64, _i64, _int, _p, _p, _f32]
lib.puro_layer_norm.argtypes = _norm_in + [_p, _i64, _p, _p, _p]
lib.puro_layer_norm_quant.argtypes = _norm_in + [_p, _i64, _p, _p, _p, _p]
lib.puro_layer_norm_quant_dual.argtypes = _norm_in + [_p, _i64, _p, _p, _i64, _p, _p, _p, _p]
lib.puro_layer_norm_backward.argtypes = [_int, _int, _p, _i64, _p, _i64, _i64, _i64, _int, _p, _p, _p, _p, _i64, _p, _p,
                                         _int, _p, _sz, _p]
lib.puro_layer_norm_backward_workspace_size.argtypes = [_i64, _i64]
lib.puro_grad_norm.argtypes = [_jobs, _int, _p, _p, _sz, _p]
lib.puro_clip_grad_norm.argtypes = [_jobs, _int, _f32, _p, _p, _sz, _p]
lib.puro_scale_by_norm.argtypes = [_jobs, _int, _f32, _p, _p]
lib.puro_grad_norm_workspace_size.argtypes = [_jobs, _int]
lib.puro_gemm_rows.argtypes = [_i64, _i64, _i64, _p, _i64, _p, _p, _i64, _p, _p, _i64, _int, _p, _sz, _p]
lib.puro_gemm_rows_workspace_size.argtypes = [_i64, _i64, _i64]
for _f in EXPORTED_OPS:
    getattr(lib, _f).restype = _sz if _f.endswith("_workspace_size") else _int

_DTYPE = {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32}


def _dtype(t, what: str) -> int:
    code = _DTYPE.get(getattr(t, "dtype", None))
    if code is None:
        raise TypeError(f"{what}: expected a bf16 or fp32 torch.Tensor")
    return code


def _kind(kind) -> int:
    if kind not in (LAYER_NORM, RMS_NORM):
        raise ValueError(f"kind {kind}: expected LAYER_NORM or RMS_NORM")
    return kind


def _matrix(x, what: str):
    """(rows, columns, row stride) of a bf16 or fp32 matrix on the current GPU with unit element stride."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{what}: expected a 2-D tensor")
    _need(x, what, x.dtype, None)
    T, C = x.shape
    return T, C, _row_stride(x)


def _row_stride(t) -> int:
    """Row stride of a checked matrix; a single row or an empty one may carry any stride."""
    T, C = t.shape
    if T <= 1:
        return max(C, 1)
    if t.stride(0) < C:
        raise ValueError(f"row stride {t.stride(0)} is smaller than a row of {C}")
    return t.stride(0)


def _vector(v, what: str, C: int):
    _need(v, what, v.dtype if isinstance(v, torch.Tensor) else None, (C,), whole=True)
    return v.data_ptr()


def _norm_inputs(x, weight, bias, eps, kind):
    """Checks and C arguments that every forward form shares."""
    xd = _dtype(x, "x")
    T, C, ldx = _matrix(x, "x")
    wd = _dtype(weight, "weight")
    pw = _vector(weight, "weight", C)
    pb = None
    if bias is not None:
        if _dtype(bias, "bias") != wd:
            raise TypeError(f"bias: dtype {bias.dtype}, expected the weight's {weight.dtype}")
        pb = _vector(bias, "bias", C)
    return T, C, [_kind(kind), xd, x.data_ptr(), T, C, ldx, wd, pw, pb, eps]


def _stats(x, T, mean, rstd, kind, make):
    """The statistics' tensors: allocated where wanted and not given, checked where given."""
    if kind == RMS_NORM:
        if mean is not None:
            raise ValueError("mean: an RMS norm has none")
    elif mean is None and make:
        mean = torch.empty(T, dtype=torch.float32, device=x.device)
    elif mean is not None:
        _need(mean, "mean", torch.float32, (T,), whole=True)
    if rstd is None:
        if make:
            rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    else:
        _need(rstd, "rstd", torch.float32, (T,), whole=True)
    return mean, rstd


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on_stream(call):
    """Give an entry point its `stream` argument: the call then runs as under torch.cuda.stream, so what it
    allocates (outputs, workspace) comes from that stream's memory and is not handed out again before the work on it
    is done.  A caller that uses such an output on another stream orders the two, as for any tensor."""
    @functools.wraps(call)
    def entry(*args, stream=None, **kw):
        if stream is None:
            return call(*args, **kw)
        with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream):
            return call(*args, **kw)
    return entry


def _out(t, what, x, dtype, shape, whole=False):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=x.device)
    return _need(t, what, dtype, shape, whole)


@_on_stream
def puro_layer_norm(x, weight, bias=None, eps: float = 1e-5, kind: int = LAYER_NORM, y=None, mean=None, rstd=None,
                    stats: bool = True):
    """x [T, C] bf16 or fp32 -> (y [T, C] of x's type, mean fp32 [T], rstd fp32 [T]): the layer or RMS norm
    of each row and the statistics its backward pass takes.  mean is None for RMS_NORM; with stats=False
    only the statistics given are written.  y may be x."""
    T, C, args = _norm_inputs(x, weight, bias, eps, kind)
    y = _out(y, "y", x, x.dtype, (T, C))
    mean, rstd = _stats(x, T, mean, rstd, kind, stats)
    _check(lib.puro_layer_norm(*args, y.data_ptr(), _row_stride(y), _ptr(mean), _ptr(rstd), _stream(None)),
           "puro_layer_norm")
    return y, mean, rstd


@_on_stream
def puro_layer_norm_quant(x, weight, bias=None, eps: float = 1e-5, kind: int = LAYER_NORM, q=None, s=None, mean=None,
                          rstd=None):
    """x [T, C] -> (q uint8 [T, C], s fp32 [C/128, T]): the norm of each row as 1x128 codes and scales
    (layouts of puro_fp8_quant_act_1x128), for any T.  mean and rstd are written where given."""
    T, C, args = _norm_inputs(x, weight, bias, eps, kind)
    q = _out(q, "q", x, torch.uint8, (T, C))
    s = _out(s, "s", x, torch.float32, (C // 128, T), True)
    mean, rstd = _stats(x, T, mean, rstd, kind, False)
    _check(lib.puro_layer_norm_quant(*args, q.data_ptr(), _row_stride(q), s.data_ptr(), _ptr(mean), _ptr(rstd),
                                     _stream(None)), "puro_layer_norm_quant")
    return q, s


@_on_stream
def puro_layer_norm_quant_dual(x, weight, bias=None, eps: float = 1e-5, kind: int = LAYER_NORM, q=None, s=None, qT=None,
                               sT=None, mean=None, rstd=None):
    """x [T, C] -> (q [T, C], s [C/128, T], qT [C, T], sT [T/128, C], mean, rstd): the norm of each row as the
    codes and scales of both orientations (layouts of puro_fp8_quant_act_dual), and its statistics."""
    T, C, args = _norm_inputs(x, weight, bias, eps, kind)
    q = _out(q, "q", x, torch.uint8, (T, C))
    s = _out(s, "s", x, torch.float32, (C // 128, T), True)
    qT = _out(qT, "qT", x, torch.uint8, (C, T))
    sT = _out(sT, "sT", x, torch.float32, (T // 128, C), True)
    mean, rstd = _stats(x, T, mean, rstd, kind, True)
    _check(lib.puro_layer_norm_quant_dual(*args, q.data_ptr(), _row_stride(q), s.data_ptr(), qT.data_ptr(),
                                          _row_stride(qT), sT.data_ptr(), _ptr(mean), _ptr(rstd), _stream(None)),
           "puro_layer_norm_quant_dual")
    return q, s, qT, sT, mean, rstd


def puro_layer_norm_backward_workspace_size(T: int, C: int) -> int:
    return lib.puro_layer_norm_backward_workspace_size(T, C)


def _workspace(workspace, need: int, device):
    """(workspace, its bytes): allocated when needed and not given."""
    if workspace is None:
        if not need:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _need(workspace, "workspace", workspace.dtype if isinstance(workspace, torch.Tensor) else None, None, whole=True)
    return workspace, workspace.numel() * workspace.element_size()


@_on_stream
def puro_layer_norm_backward(dy, x, weight, mean, rstd, kind: int = LAYER_NORM, dx=None, dweight=None, dbias=None,
                             with_bias: bool = True, accumulate: bool = False, workspace=None):
    """(dx [T, C] of x's type, dweight fp32 [C], dbias fp32 [C] or None): the backward pass of the norm, from
    the statistics of the forward pass (mean is None for RMS_NORM).  accumulate adds to the dweight and dbias given.
    dx may be dy or x."""
    xd = _dtype(x, "x")
    T, C, ldx = _matrix(x, "x")
    _need(dy, "dy", x.dtype, (T, C))
    wd = _dtype(weight, "weight")
    pw = _vector(weight, "weight", C)
    if _kind(kind) == LAYER_NORM:
        _need(mean, "mean", torch.float32, (T,), whole=True)
    elif mean is not None:
        raise ValueError("mean: an RMS norm has none")
    _need(rstd, "rstd", torch.float32, (T,), whole=True)
    if accumulate and (dweight is None or (with_bias and dbias is None)):
        raise ValueError("accumulate: needs the gradients it adds to")
    dx = _out(dx, "dx", x, x.dtype, (T, C))
    dweight = _out(dweight, "dweight", x, torch.float32, (C,), True)
    if with_bias or dbias is not None:
        dbias = _out(dbias, "dbias", x, torch.float32, (C,), True)
    workspace, wbytes = _workspace(workspace, lib.puro_layer_norm_backward_workspace_size(T, C), x.device)
    _check(lib.puro_layer_norm_backward(kind, xd, dy.data_ptr(), _row_stride(dy), x.data_ptr(), ldx, T, C, wd, pw,
                                        _ptr(mean), rstd.data_ptr(), dx.data_ptr(), _row_stride(dx), dweight.data_ptr(),
                                        _ptr(dbias), 1 if accumulate else 0, _ptr(workspace), wbytes,
                                        _stream(None)), "puro_layer_norm_backward")
    return dx, dweight, dbias


def _grad_jobs(grads, outs):
    """The job array of a list of gradients, and the device they share."""
    if outs is not None and len(outs) != len(grads):
        raise ValueError(f"outs: {len(outs)} tensors for {len(grads)} gradients")
    jobs = (GradJob * max(len(grads), 1))()
    for i, g in enumerate(grads):
        code = _dtype(g, f"grads[{i}]")
        _need(g, f"grads[{i}]", g.dtype, None, whole=True)
        src = dst = g.data_ptr()
        if outs is not None:
            dst = _need(outs[i], f"outs[{i}]", g.dtype, g.shape, whole=True).data_ptr()
        job = jobs[i]
        job.src, job.dst, job.n, job.dtype = src, dst, g.numel(), code
    return jobs


def _norm_tensor(norm):
    if norm is None:
        return torch.empty((), dtype=torch.float32, device="cuda")
    _need(norm, "norm", torch.float32, None, whole=True)
    if norm.numel() != 1:
        raise ValueError("norm: expected one value")
    return norm


@_on_stream
def puro_grad_norm(grads, norm=None, workspace=None):
    """norm (fp32, one value, on the GPU): the square root of the sum of all squares of a list of contiguous
    bf16 or fp32 tensors."""
    grads = list(grads)
    jobs = _grad_jobs(grads, None)
    norm = _norm_tensor(norm)
    workspace, wbytes = _workspace(workspace, lib.puro_grad_norm_workspace_size(jobs, len(grads)), norm.device)
    _check(lib.puro_grad_norm(jobs, len(grads), norm.data_ptr(), _ptr(workspace), wbytes, _stream(None)),
           "puro_grad_norm")
    return norm


@_on_stream
def puro_clip_grad_norm(grads, max_norm: float, outs=None, norm=None, workspace=None):
    """(norm, outs): the global norm of a list of contiguous bf16 or fp32 tensors, and the tensors times
    min(1, max_norm / (norm + 1e-6)) -- in place (outs is then grads), or into the tensors given as outs."""
    grads = list(grads)
    jobs = _grad_jobs(grads, outs)
    norm = _norm_tensor(norm)
    workspace, wbytes = _workspace(workspace, lib.puro_grad_norm_workspace_size(jobs, len(grads)), norm.device)
    _check(lib.puro_clip_grad_norm(jobs, len(grads), max_norm, norm.data_ptr(), _ptr(workspace), wbytes,
                                   _stream(None)), "puro_clip_grad_norm")
    return norm, grads if outs is None else outs


@_on_stream
def puro_scale_by_norm(grads, max_norm: float, norm, outs=None):
    """The tensors times min(1, max_norm / (norm + 1e-6)) with a norm already on the GPU (for instance joined
    over processes); in place, or into outs.  Returns the tensors written."""
    grads = list(grads)
    jobs = _grad_jobs(grads, outs)
    if norm is None:
        raise ValueError("norm: the scaling needs the norm's tensor")
    norm = _norm_tensor(norm)
    _check(lib.puro_scale_by_norm(jobs, len(grads), max_norm, norm.data_ptr(), _stream(None)), "puro_scale_by_norm")
    return grads if outs is None else outs


def puro_gemm_rows_workspace_size(M: int, N: int, K: int) -> int:
    return lib.puro_gemm_rows_workspace_size(M, N, K)


@_on_stream
def puro_gemm_rows(A, sA, B, sB, C=None, out_dtype: int = OUT_BF16, workspace=None):
    """C [M, N] = blockwise-scaled FP8 product of A [M, K] (sA fp32 [K/128, M]) and B [N, K] (sB fp32
    [N/128, K/128]) for any number of rows M; see puro_ops.h."""
    for t, what in ((A, "A"), (B, "B")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{what}: expected a 2-D tensor")
    M, K = A.shape
    N, KB = B.shape
    if KB != K:
        raise ValueError(f"A [{M}, {K}] and B [{N}, {KB}] differ in the contraction length")
    _need(A, "A", torch.uint8, None)
    _need(B, "B", torch.uint8, None)
    _need(sA, "sA", torch.float32, (K // 128, M), whole=True)
    _need(sB, "sB", torch.float32, (N // 128, K // 128), whole=True)
    if out_dtype not in (OUT_BF16, OUT_FP32):
        raise ValueError(f"out_dtype {out_dtype}: expected OUT_BF16 or OUT_FP32")
    C = _out(C, "C", A, torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32, (M, N))
    workspace, wbytes = _workspace(workspace, lib.puro_gemm_rows_workspace_size(M, N, K), A.device)
    _check(lib.puro_gemm_rows(M, N, K, A.data_ptr(), _row_stride(A), sA.data_ptr(), B.data_ptr(), _row_stride(B),
                              sB.data_ptr(), C.data_ptr(), _row_stride(C), out_dtype, _ptr(workspace), wbytes,
                              _stream(None)), "puro_gemm_rows")
    return C
