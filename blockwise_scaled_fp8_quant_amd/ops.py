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

from . import OUT_BF16, OUT_FP32, _check, _i64, _int, _need, _p, _sz, lib

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


_jobs = _p     # a host array of GradJob
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
_f32t, _u8t = torch.float32, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream    # the current stream's handle, without the wrapper's checks


def _device() -> int:
    """The current GPU's index; one that no tensor has where there is no GPU (every check then refuses)."""
    try:
        return torch._C._cuda_getDevice()
    except RuntimeError:
        return -2


# The checks below are the package's (_need), with the passing case first: a decode step calls these entry points
# thousands of times a second, and its time is the host's.  (Two further differences: a dimension of one element may
# carry any stride, as in is_contiguous, and rows may be any distance apart that is no less than their length.)
def _whole(t, what: str, dtype, shape, dev: int) -> int:
    """Data pointer of a contiguous tensor of `dtype` (None: any) and `shape` (None: any) on GPU `dev`."""
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and (dtype is None or t.dtype is dtype)
            and (shape is None or t.shape == shape) and t.is_contiguous()):
        return t.data_ptr()
    _need(t, what, getattr(t, "dtype", None) if dtype is None else dtype, shape, whole=True)
    raise ValueError(f"{what}: must be contiguous")


def _rows_of(t, what: str, dtype, shape, dev: int) -> int:
    """Row stride of a matrix of `dtype` and `shape` (None: any two dimensions) on GPU `dev`."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{what}: expected a 2-D tensor")
    T, C = t.shape
    if t.get_device() != dev or t.dtype is not dtype or (shape is not None and t.shape != shape):
        _need(t, what, dtype, shape)
    ld, step = t.stride()
    if step != 1 and C > 1 and T > 0:
        raise ValueError(f"{what}: rows must have unit element stride (got strides {t.stride()})")
    if T <= 1 or C == 0:
        return C if C > 0 else 1                    # a single row's stride says nothing
    if ld < C:
        raise ValueError(f"{what}: row stride {ld} is smaller than a row of {C}")
    return ld


def _dtype(t, what: str) -> int:
    code = _DTYPE.get(getattr(t, "dtype", None))
    if code is None:
        raise TypeError(f"{what}: expected a bf16 or fp32 torch.Tensor")
    return code


def _kind(kind) -> int:
    if kind not in (LAYER_NORM, RMS_NORM):
        raise ValueError(f"kind {kind}: expected LAYER_NORM or RMS_NORM")
    return kind


def _norm_inputs(x, weight, bias, eps, kind, dev):
    """Checks and C arguments that every forward form shares."""
    xd = _dtype(x, "x")
    ldx = _rows_of(x, "x", x.dtype, None, dev)
    T, C = x.shape
    wd = _dtype(weight, "weight")
    pw = _whole(weight, "weight", weight.dtype, (C,), dev)
    pb = None if bias is None else _whole(bias, "bias", weight.dtype, (C,), dev)
    return T, C, (_kind(kind), xd, x.data_ptr(), T, C, ldx, wd, pw, pb, eps)


def _stats(T, mean, rstd, kind, make, dev):
    """The statistics' tensors (allocated where wanted and not given) and their pointers."""
    pm = pr = None
    if mean is not None:
        if kind == RMS_NORM:
            raise ValueError("mean: an RMS norm has none")
        pm = _whole(mean, "mean", _f32t, (T,), dev)
    elif make and kind == LAYER_NORM:
        mean = torch.empty(T, dtype=_f32t, device="cuda")
        pm = mean.data_ptr()
    if rstd is not None:
        pr = _whole(rstd, "rstd", _f32t, (T,), dev)
    elif make:
        rstd = torch.empty(T, dtype=_f32t, device="cuda")
        pr = rstd.data_ptr()
    return mean, rstd, pm, pr


def _out_rows(t, what, dtype, shape, dev):
    """An output matrix and its row stride."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device="cuda"), shape[1] or 1
    return t, _rows_of(t, what, dtype, shape, dev)


def _out_whole(t, what, dtype, shape, dev):
    """A contiguous output and its pointer."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device="cuda")
        return t, t.data_ptr()
    return t, _whole(t, what, dtype, shape, dev)


def _workspace(workspace, need: int, dev):
    """(workspace, its pointer, its bytes): allocated when needed and not given."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=_u8t, device="cuda")
        return workspace, workspace.data_ptr(), need
    return workspace, _whole(workspace, "workspace", None, None, dev), workspace.numel() * workspace.element_size()


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


@_on_stream
def puro_layer_norm(x, weight, bias=None, eps: float = 1e-5, kind: int = LAYER_NORM, y=None, mean=None, rstd=None,
                    stats: bool = True):
    """x [T, C] bf16 or fp32 -> (y [T, C] of x's type, mean fp32 [T], rstd fp32 [T]): the layer or RMS norm
    of each row and the statistics its backward pass takes.  mean is None for RMS_NORM; with stats=False
    only the statistics given are written.  y may be x."""
    dev = _device()
    T, C, args = _norm_inputs(x, weight, bias, eps, kind, dev)
    y, ldy = _out_rows(y, "y", x.dtype, (T, C), dev)
    mean, rstd, pm, pr = _stats(T, mean, rstd, kind, stats, dev)
    _check(lib.puro_layer_norm(*args, y.data_ptr(), ldy, pm, pr, _raw_stream(dev)), "puro_layer_norm")
    return y, mean, rstd


@_on_stream
def puro_layer_norm_quant(x, weight, bias=None, eps: float = 1e-5, kind: int = LAYER_NORM, q=None, s=None, mean=None,
                          rstd=None):
    """x [T, C] -> (q uint8 [T, C], s fp32 [C/128, T]): the norm of each row as 1x128 codes and scales
    (layouts of puro_fp8_quant_act_1x128), for any T.  mean and rstd are written where given."""
    dev = _device()
    T, C, args = _norm_inputs(x, weight, bias, eps, kind, dev)
    q, ldq = _out_rows(q, "q", _u8t, (T, C), dev)
    s, ps = _out_whole(s, "s", _f32t, (C // 128, T), dev)
    _, _, pm, pr = _stats(T, mean, rstd, kind, False, dev)
    _check(lib.puro_layer_norm_quant(*args, q.data_ptr(), ldq, ps, pm, pr, _raw_stream(dev)), "puro_layer_norm_quant")
    return q, s


@_on_stream
def puro_layer_norm_quant_dual(x, weight, bias=None, eps: float = 1e-5, kind: int = LAYER_NORM, q=None, s=None, qT=None,
                               sT=None, mean=None, rstd=None):
    """x [T, C] -> (q [T, C], s [C/128, T], qT [C, T], sT [T/128, C], mean, rstd): the norm of each row as the
    codes and scales of both orientations (layouts of puro_fp8_quant_act_dual), and its statistics."""
    dev = _device()
    T, C, args = _norm_inputs(x, weight, bias, eps, kind, dev)
    q, ldq = _out_rows(q, "q", _u8t, (T, C), dev)
    s, ps = _out_whole(s, "s", _f32t, (C // 128, T), dev)
    qT, ldqT = _out_rows(qT, "qT", _u8t, (C, T), dev)
    sT, psT = _out_whole(sT, "sT", _f32t, (T // 128, C), dev)
    mean, rstd, pm, pr = _stats(T, mean, rstd, kind, True, dev)
    _check(lib.puro_layer_norm_quant_dual(*args, q.data_ptr(), ldq, ps, qT.data_ptr(), ldqT, psT, pm, pr,
                                          _raw_stream(dev)), "puro_layer_norm_quant_dual")
    return q, s, qT, sT, mean, rstd


def puro_layer_norm_backward_workspace_size(T: int, C: int) -> int:
    return lib.puro_layer_norm_backward_workspace_size(T, C)


@_on_stream
def puro_layer_norm_backward(dy, x, weight, mean, rstd, kind: int = LAYER_NORM, dx=None, dweight=None, dbias=None,
                             with_bias: bool = True, accumulate: bool = False, workspace=None):
    """(dx [T, C] of x's type, dweight fp32 [C], dbias fp32 [C] or None): the backward pass of the norm, from
    the statistics of the forward pass (mean is None for RMS_NORM).  accumulate adds to the dweight and dbias given.
    dx may be dy or x."""
    dev = _device()
    xd = _dtype(x, "x")
    ldx = _rows_of(x, "x", x.dtype, None, dev)
    T, C = x.shape
    lddy = _rows_of(dy, "dy", x.dtype, (T, C), dev)
    wd = _dtype(weight, "weight")
    pw = _whole(weight, "weight", weight.dtype, (C,), dev)
    pm = None
    if _kind(kind) == LAYER_NORM:
        pm = _whole(mean, "mean", _f32t, (T,), dev)
    elif mean is not None:
        raise ValueError("mean: an RMS norm has none")
    pr = _whole(rstd, "rstd", _f32t, (T,), dev)
    if accumulate and (dweight is None or (with_bias and dbias is None)):
        raise ValueError("accumulate: needs the gradients it adds to")
    dx, lddx = _out_rows(dx, "dx", x.dtype, (T, C), dev)
    dweight, pdw = _out_whole(dweight, "dweight", _f32t, (C,), dev)
    pdb = None
    if with_bias or dbias is not None:
        dbias, pdb = _out_whole(dbias, "dbias", _f32t, (C,), dev)
    workspace, pws, wbytes = _workspace(workspace, lib.puro_layer_norm_backward_workspace_size(T, C), dev)
    _check(lib.puro_layer_norm_backward(kind, xd, dy.data_ptr(), lddy, x.data_ptr(), ldx, T, C, wd, pw, pm, pr,
                                        dx.data_ptr(), lddx, pdw, pdb, 1 if accumulate else 0, pws, wbytes,
                                        _raw_stream(dev)), "puro_layer_norm_backward")
    return dx, dweight, dbias


def _grad_jobs(grads, outs, dev):
    """The job array (puro_grad_job) of a list of gradients: four 64-bit words each."""
    words = []
    if outs is not None and len(outs) != len(grads):
        raise ValueError(f"outs: {len(outs)} tensors for {len(grads)} gradients")
    for i, g in enumerate(grads):
        dtype = getattr(g, "dtype", None)
        code = _DTYPE.get(dtype)
        if code is None:
            _dtype(g, f"grads[{i}]")
        # (the tests of _whole, inline: a model has hundreds of gradients)
        if g.get_device() != dev or not g.is_contiguous():
            _whole(g, f"grads[{i}]", dtype, None, dev)
        src = dst = g.data_ptr()
        if outs is not None:
            o = outs[i]
            if not (isinstance(o, torch.Tensor) and o.dtype is dtype and o.get_device() == dev and o.shape == g.shape
                    and o.is_contiguous()):
                _whole(o, f"outs[{i}]", dtype, g.shape, dev)
            dst = o.data_ptr()
        words += (src, dst, g.numel(), code)
    return (_i64 * max(len(words), 4))(*words)


def _norm_tensor(norm, dev):
    if norm is None:
        return torch.empty((), dtype=_f32t, device="cuda")
    _whole(norm, "norm", _f32t, None, dev)
    if norm.numel() != 1:
        raise ValueError("norm: expected one value")
    return norm


@_on_stream
def puro_grad_norm(grads, norm=None, workspace=None):
    """norm (fp32, one value, on the GPU): the square root of the sum of all squares of a list of contiguous
    bf16 or fp32 tensors."""
    dev = _device()
    grads = list(grads)
    jobs = _grad_jobs(grads, None, dev)
    norm = _norm_tensor(norm, dev)
    workspace, pws, wbytes = _workspace(workspace, lib.puro_grad_norm_workspace_size(jobs, len(grads)), dev)
    _check(lib.puro_grad_norm(jobs, len(grads), norm.data_ptr(), pws, wbytes, _raw_stream(dev)), "puro_grad_norm")
    return norm


@_on_stream
def puro_clip_grad_norm(grads, max_norm: float, outs=None, norm=None, workspace=None):
    """(norm, outs): the global norm of a list of contiguous bf16 or fp32 tensors, and the tensors times
    min(1, max_norm / (norm + 1e-6)) -- in place (outs is then grads), or into the tensors given as outs."""
    dev = _device()
    grads = list(grads)
    jobs = _grad_jobs(grads, outs, dev)
    norm = _norm_tensor(norm, dev)
    workspace, pws, wbytes = _workspace(workspace, lib.puro_grad_norm_workspace_size(jobs, len(grads)), dev)
    _check(lib.puro_clip_grad_norm(jobs, len(grads), max_norm, norm.data_ptr(), pws, wbytes, _raw_stream(dev)),
           "puro_clip_grad_norm")
    return norm, grads if outs is None else outs


@_on_stream
def puro_scale_by_norm(grads, max_norm: float, norm, outs=None):
    """The tensors times min(1, max_norm / (norm + 1e-6)) with a norm already on the GPU (for instance joined
    over processes); in place, or into outs.  Returns the tensors written."""
    if norm is None:
        raise ValueError("norm: the scaling needs the norm's tensor")
    dev = _device()
    grads = list(grads)
    jobs = _grad_jobs(grads, outs, dev)
    norm = _norm_tensor(norm, dev)
    _check(lib.puro_scale_by_norm(jobs, len(grads), max_norm, norm.data_ptr(), _raw_stream(dev)), "puro_scale_by_norm")
    return grads if outs is None else outs


def puro_gemm_rows_workspace_size(M: int, N: int, K: int) -> int:
    return lib.puro_gemm_rows_workspace_size(M, N, K)


@_on_stream
def puro_gemm_rows(A, sA, B, sB, C=None, out_dtype: int = OUT_BF16, workspace=None):
    """C [M, N] = blockwise-scaled FP8 product of A [M, K] (sA fp32 [K/128, M]) and B [N, K] (sB fp32
    [N/128, K/128]) for any number of rows M; see puro_ops.h."""
    dev = _device()
    lda = _rows_of(A, "A", _u8t, None, dev)
    ldb = _rows_of(B, "B", _u8t, None, dev)
    M, K = A.shape
    N, KB = B.shape
    if KB != K:
        raise ValueError(f"A [{M}, {K}] and B [{N}, {KB}] differ in the contraction length")
    psA = _whole(sA, "sA", _f32t, (K // 128, M), dev)
    psB = _whole(sB, "sB", _f32t, (N // 128, K // 128), dev)
    if out_dtype not in (OUT_BF16, OUT_FP32):
        raise ValueError(f"out_dtype {out_dtype}: expected OUT_BF16 or OUT_FP32")
    C, ldc = _out_rows(C, "C", torch.bfloat16 if out_dtype == OUT_BF16 else _f32t, (M, N), dev)
    need = lib.puro_gemm_rows_workspace_size(M, N, K) if out_dtype == OUT_BF16 else 0
    workspace, pws, wbytes = _workspace(workspace, need, dev)
    _check(lib.puro_gemm_rows(M, N, K, A.data_ptr(), lda, psA, B.data_ptr(), ldb, psB, C.data_ptr(), ldc, out_dtype, pws,
                              wbytes, _raw_stream(dev)), "puro_gemm_rows")
    return C
