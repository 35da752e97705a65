"""Host-side checks of include/puro_ops.h (no GPU, no kernel launched): the header, the binding and the library
name the same entry points; every call below has an invalid argument or an empty shape, so the library returns
before any HIP call."""
import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest

import blockwise_scaled_fp8_quant_amd as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "puro_ops.h")
OK, NULLPTR, SHAPE, ALIGN, LD, MODE, DTYPE, WORKSPACE, UNSUP, ARG = 0, -1, -2, -3, -4, -5, -6, -7, -9, -10
A16, MIS = 0x10000, 0x10008       # never dereferenced: validation fails first
BF16, FP32 = 0, 1


def declared():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(puro_\w+)\s*\(", src)))


def test_header_binding_and_library_agree():
    assert sorted(P.EXPORTED_OPS) == declared()
    out = subprocess.run(["nm", "-D", "--defined-only", P.LIB_PATH], capture_output=True, text=True).stdout
    for name in declared():
        assert re.search(rf"\bT {name}\b", out), name
        assert hasattr(P, name) or name == "puro_grad_norm_workspace_size"
    assert P.puro_fp8_strerror(ARG) != "unknown status"


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_header_is_strict_c11(tmp_path):
    src = tmp_path / "p.c"
    src.write_text('#include "puro_ops.h"\nint main(void) { puro_grad_job j = {0}; return j.n != 0; }\n')
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                        os.path.join(ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "p.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def norm(kind=0, xd=BF16, x=A16, T=4, C=256, ldx=256, wd=BF16, w=A16, b=A16, eps=1e-5, y=A16, ldy=256, mean=A16,
         rstd=A16):
    return P.lib.puro_layer_norm(kind, xd, x, T, C, ldx, wd, w, b, eps, y, ldy, mean, rstd, None)


def test_norm_refusals():
    assert norm(T=0) == OK and norm(C=0) == OK and norm(T=0, x=None, y=None) == OK
    assert norm(kind=2) == MODE and norm(xd=2) == DTYPE and norm(wd=-1) == DTYPE
    assert norm(T=-1) == SHAPE and norm(C=-1) == SHAPE
    for eps in (-1e-5, math.nan, math.inf):
        assert norm(eps=eps) == ARG
    assert norm(kind=1) == ARG                                   # an RMS norm has no mean
    assert norm(x=None) == NULLPTR and norm(w=None) == NULLPTR and norm(y=None) == NULLPTR
    assert norm(x=A16 + 1) == ALIGN and norm(y=A16 + 1) == ALIGN and norm(xd=FP32, x=A16 + 2) == ALIGN
    assert norm(wd=FP32, w=A16 + 2) == ALIGN and norm(mean=A16 + 2) == ALIGN and norm(rstd=A16 + 1) == ALIGN
    assert norm(ldx=255) == LD and norm(ldy=255) == LD
    assert norm(C=16385, ldx=16385, ldy=16385) == UNSUP


def quant(T=4, C=256, x=A16, ldx=256, q=A16, ldq=256, s=A16, kind=0, mean=None, rstd=None, w=A16, b=None, eps=1e-5):
    return P.lib.puro_layer_norm_quant(kind, BF16, x, T, C, ldx, BF16, w, b, eps, q, ldq, s, mean, rstd, None)


def test_norm_quant_refusals():
    assert quant(T=0) == OK and quant(C=0) == OK
    assert quant(C=200) == SHAPE and quant(T=-1) == SHAPE
    assert quant(q=None) == NULLPTR and quant(s=None) == NULLPTR and quant(x=None) == NULLPTR
    assert quant(x=MIS) == ALIGN and quant(q=MIS) == ALIGN and quant(s=MIS) == ALIGN and quant(w=MIS) == ALIGN
    assert quant(b=MIS) == ALIGN
    assert quant(ldx=128) == LD and quant(ldx=260) == LD and quant(ldq=264) == LD and quant(ldq=128) == LD
    assert quant(kind=1, mean=A16) == ARG and quant(eps=-1.0) == ARG
    assert quant(C=16512, ldx=16512, ldq=16512) == UNSUP


def dual(T=256, C=256, q=A16, s=A16, qT=A16, ldqT=256, sT=A16, mean=A16, rstd=A16, kind=0, ldq=256):
    return P.lib.puro_layer_norm_quant_dual(kind, BF16, A16, T, C, max(C, 1), BF16, A16, None, 1e-5, q, ldq, s, qT, ldqT, sT,
                                            mean, rstd, None)


def test_norm_quant_dual_refusals():
    assert dual(T=0) == OK and dual(C=0) == OK
    assert dual(T=100) == SHAPE and dual(C=64) == SHAPE and dual(T=-128) == SHAPE
    for a in ("q", "s", "qT", "sT", "rstd", "mean"):
        assert dual(**{a: None}) == NULLPTR, a
    for a in ("q", "s", "qT", "sT"):
        assert dual(**{a: MIS}) == ALIGN, a
    assert dual(ldqT=128) == LD and dual(ldqT=264) == LD and dual(ldq=264) == LD
    assert dual(kind=1) == ARG and dual(kind=1, mean=None, rstd=None) == NULLPTR


def bwd(kind=0, T=64, C=256, dy=A16, x=A16, ld=256, w=A16, mean=A16, rstd=A16, dx=A16, dw=A16, db=A16, acc=0, ws=A16,
        wb=1 << 30, xd=BF16, lddx=None):
    return P.lib.puro_layer_norm_backward(kind, xd, dy, ld, x, ld, T, C, BF16, w, mean, rstd, dx,
                                          ld if lddx is None else lddx, dw, db, acc, ws, wb, None)


def test_norm_backward_refusals():
    assert bwd(C=0) == OK and bwd(T=0, acc=1) == OK
    assert bwd(kind=3) == MODE and bwd(xd=7) == DTYPE and bwd(T=-1) == SHAPE
    assert bwd(acc=2) == ARG and bwd(kind=1) == ARG
    for a in ("dy", "x", "w", "mean", "rstd", "dx", "dw"):
        assert bwd(**{a: None}) == NULLPTR, a
    assert bwd(x=A16 + 1) == ALIGN and bwd(dw=A16 + 2) == ALIGN and bwd(mean=A16 + 1) == ALIGN
    assert bwd(ld=255) == LD and bwd(lddx=255) == LD
    assert bwd(C=16385, ld=16385) == UNSUP
    need = P.puro_layer_norm_backward_workspace_size(16384, 2048)
    assert need > 0
    assert bwd(T=16384, C=2048, ld=2048, wb=need - 1) == WORKSPACE and bwd(T=16384, C=2048, ld=2048, ws=None) == WORKSPACE
    assert bwd(T=16384, C=2048, ld=2048, ws=MIS) == ALIGN
    assert P.puro_layer_norm_backward_workspace_size(0, 2048) == 0
    assert P.puro_layer_norm_backward_workspace_size(1, 2048) == 0
    assert P.puro_layer_norm_backward_workspace_size(8, 1 << 20) == 0


def jobs(*js):
    return (P.GradJob * max(len(js), 1))(*[P.GradJob(*j) for j in js])


def clip(js, n=None, max_norm=1.0, norm=A16, ws=A16, wb=1 << 20):
    return P.lib.puro_clip_grad_norm(jobs(*js), len(js) if n is None else n, max_norm, norm, ws, wb, None)


def test_clip_refusals():
    good = (A16, A16, 100, FP32)
    for m in (-1.0, math.nan):
        assert clip([good], max_norm=m) == ARG
        assert P.lib.puro_scale_by_norm(jobs(good), 1, m, A16, None) == ARG
    assert clip([good], n=-1) == SHAPE and clip([(A16, A16, -1, FP32)]) == SHAPE
    assert clip([(A16, A16, 100, 3)]) == DTYPE
    assert clip([(None, A16, 100, FP32)]) == NULLPTR and clip([(A16, None, 100, FP32)]) == NULLPTR
    assert clip([good], norm=None) == NULLPTR and clip([good], norm=A16 + 2) == ALIGN
    assert clip([(A16 + 2, A16, 100, FP32)]) == ALIGN and clip([(A16 + 2, A16 + 1, 100, BF16)]) == ALIGN
    assert clip([good], ws=None) == WORKSPACE and clip([good], wb=4) == WORKSPACE and clip([good], ws=MIS) == ALIGN
    assert P.lib.puro_clip_grad_norm(None, 1, 1.0, A16, A16, 1 << 20, None) == NULLPTR
    assert P.lib.puro_scale_by_norm(jobs(good), 1, 1.0, None, None) == NULLPTR


def test_clip_refuses_overlaps():
    B = A16 + 4096
    same = (A16, A16, 100, FP32)
    assert clip([same, same]) == ARG                                    # one gradient listed twice
    assert clip([same, (A16 + 396, A16 + 396, 100, FP32)]) == ARG       # the last element is shared
    assert clip([(A16, B, 100, FP32), (B + 396, B + 4096, 100, FP32)]) == ARG    # an output over another's input
    assert clip([(A16, A16 + 4, 100, FP32)]) == ARG                     # an output shifted over its own input
    # two inputs may overlap; side by side is fine: these calls get as far as the workspace
    assert clip([(A16, B, 100, FP32), (A16, B + 400, 100, FP32)], ws=None) == WORKSPACE
    assert clip([same, (A16 + 400, A16 + 400, 100, FP32)], ws=None) == WORKSPACE


def test_rows_refuses_more_columns_than_a_launch_holds():
    """Eight threads to a column, counted in 32 bits."""
    N = 1 << 29
    assert rows(N=N, ldc=N) == UNSUP and rows(N=N - 128, ldc=N, M=1 << 31) == UNSUP


def test_clip_refuses_a_norm_or_workspace_inside_a_tensor():
    """Both are written while other workgroups read the tensors."""
    far, ws = A16 + (1 << 20), A16 + (2 << 20)
    src_dst = (A16, A16 + 4096, 100, FP32)
    for at in (A16, A16 + 396, A16 + 4096, A16 + 4096 + 396):
        assert clip([src_dst], norm=at, ws=ws) == ARG
        assert P.lib.puro_scale_by_norm(jobs(src_dst), 1, 1.0, at, None) == ARG
    for at in (A16, A16 + 384, A16 + 4096):                             # a workspace of one value, 8 bytes
        assert clip([src_dst], norm=far, ws=at) == ARG
    in_place = (A16 + 4, A16 + 4, 100, FP32)                            # the workspace's second half is its first element
    assert clip([in_place], norm=far, ws=A16) == ARG
    assert P.lib.puro_grad_norm(jobs((A16 + 4, None, 100, FP32)), 1, far, A16, 1 << 20, None) == ARG


def test_clip_refuses_a_norm_inside_the_workspace():
    """The norm is written while other workgroups still read the partial sums, and so do the launches of longer lists."""
    ws = A16 + (2 << 20)
    many = [(A16 + 16 * i, A16 + 16 * i, 4, FP32) for i in range(300)]          # three launches, 300 partial sums
    for at in (ws, ws + 4, ws + 8 * 300 - 4):
        assert clip(many, norm=at, ws=ws) == ARG
    assert clip([(A16, A16, 100, FP32)], norm=ws + 4, ws=ws) == ARG


def test_grad_workspace_size():
    size = P.lib.puro_grad_norm_workspace_size
    assert size(jobs(), 0) == 0 and size(jobs((A16, None, 0, FP32)), 1) == 0
    assert size(jobs((A16, None, 1, FP32)), 1) == 8
    # 4096 fp32 elements make one step of a workgroup; one more needs a second, and so does a start off 16 bytes
    assert size(jobs((A16, None, 4096, FP32)), 1) == 8 and size(jobs((A16, None, 4097, FP32)), 1) == 16
    assert size(jobs((A16 + 4, None, 4096, FP32)), 1) == 16
    assert size(jobs(*[(A16, None, 1, BF16)] * 300), 300) == 300 * 8
    assert size(jobs((A16, None, 1, 9)), 1) == 0


def rows(M=3, N=256, K=256, A=A16, lda=256, sA=A16, B=A16, ldb=256, sB=A16, C=A16, ldc=256, od=BF16, ws=None, wb=0):
    return P.lib.puro_gemm_rows(M, N, K, A, lda, sA, B, ldb, sB, C, ldc, od, ws, wb, None)


def test_rows_refusals():
    assert rows(M=0) == OK and rows(N=0) == OK
    assert rows(M=-1) == SHAPE and rows(N=200) == SHAPE and rows(K=100) == SHAPE
    assert rows(od=2) == DTYPE
    for a in ("A", "sA", "B", "sB", "C"):
        assert rows(**{a: None}) == NULLPTR, a
    for a in ("A", "B", "C"):
        assert rows(**{a: MIS}) == ALIGN, a
    assert rows(sA=A16 + 2) == ALIGN and rows(sB=A16 + 1) == ALIGN
    assert rows(lda=128) == LD and rows(ldb=264) == LD and rows(ldc=128) == LD and rows(ldc=260) == LD
    assert rows(M=1 << 32) == UNSUP and rows(N=1 << 30, ldc=1 << 30) == UNSUP and rows(lda=(1 << 29) + 16) == UNSUP and rows(ldb=(1 << 29) + 16) == UNSUP
    # a long product whose leading rows the blockwise GEMM splits over the contraction wants its workspace for bf16
    big = dict(M=1030, N=512, K=1 << 14, lda=1 << 14, ldb=1 << 14, ldc=512)
    need = P.puro_gemm_rows_workspace_size(1030, 512, 1 << 14)
    assert need == P.puro_fp8_gemm_workspace_size(P.FWD, 1024, 512, 1 << 14) > 0
    assert rows(**big) == WORKSPACE and rows(**big, ws=A16, wb=need - 1) == WORKSPACE and rows(**big, ws=MIS, wb=need) == ALIGN
    assert P.puro_gemm_rows_workspace_size(0, 128, 128) == 0 and P.puro_gemm_rows_workspace_size(-1, 128, 128) == 0


def test_binding_refuses_what_the_library_cannot_see():
    import torch
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        P.puro_layer_norm(x, w)                                          # host tensors
    with pytest.raises(TypeError):
        P.puro_layer_norm(x.half(), w)
    with pytest.raises(TypeError):
        P.puro_clip_grad_norm([x.double()], 1.0)
    with pytest.raises(ValueError):
        P.puro_clip_grad_norm([x], 1.0, outs=[])
    with pytest.raises(ValueError):
        P.puro_scale_by_norm([], 1.0, None)
    with pytest.raises(ValueError):
        P.puro_gemm_rows(x, x, x, x)
    with pytest.raises(ValueError):
        P.puro_gemm_rows(x[0], x, x, x)


def test_a_stream_is_taken_for_what_it_is(monkeypatch):
    """The handle 0 is the default stream's, any other an external stream's; a stream object is itself."""
    import contextlib
    import torch
    from blockwise_scaled_fp8_quant_amd import ops
    ran = []

    @contextlib.contextmanager
    def stream(s):
        ran.append(s)
        yield
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: "the default stream")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: ("external", h))
    for given, runs in ((0, "the default stream"), (4096, ("external", 4096)), ("an object", "an object")):
        assert ops._on(given, lambda a, b: (a, b))(1, 2) == (1, 2) and ran.pop() == runs
    assert ops._on(None, len) is len and not ran


def test_captured_linear_steps_are_checked(monkeypatch):
    """Every differentiable call made while a graph is recorded is checked before its forward pass starts."""
    import torch
    from blockwise_scaled_fp8_quant_amd import linear, norm

    class Stop(Exception):
        pass

    def check(leaves):
        raise Stop(len(leaves))
    monkeypatch.setattr(linear, "check_capture", check)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)

    class OnGpu(torch.Tensor):
        is_cuda = True
    x = torch.zeros((128, 128), dtype=torch.bfloat16).as_subclass(OnGpu)
    lin, n, both = linear.Fp8Linear(128, 128), norm.Norm(128), norm.Fp8NormLinear(128, 128)
    for call in (lambda: lin(x), lambda: linear.fp8_linear(x, lin.weight), lambda: n(x), lambda: both(x),
                 lambda: norm.layer_norm(x, n.weight, n.bias), lambda: norm.rms_norm(x, n.weight)):
        with pytest.raises(Stop):
            call()


def test_norm_backward_workgroups_grow_with_the_rows():
    """No team takes more than 64 times 64 rows: 8 bytes of partial sums per column and workgroup, 512 threads each, of
    which one row takes 16 to 512 by its width."""
    for C, lanes in ((8, 16), (128, 16), (200, 32), (1000, 64), (2000, 128), (4096, 256), (4104, 512), (16384, 512)):
        teams = 512 // lanes
        for T in (1000, 16384, 262145, 1 << 20, (1 << 20) + 1, 10 ** 7, 1 << 32):
            blocks = max(P.puro_layer_norm_backward_workspace_size(T, C) // (8 * C), 1)
            assert blocks * teams * 4096 >= T and blocks * 512 < 1 << 32
            assert blocks <= 256 or T > 256 * 4096 * teams


def test_rows_workspace_follows_the_leading_rows():
    """The blockwise GEMM's workspace for the rows that it takes: 256 and more from 2^33 multiplications, 128 from 2^34."""
    size, gemm = P.puro_gemm_rows_workspace_size, lambda M, N, K: P.puro_fp8_gemm_workspace_size(P.FWD, M, N, K)
    assert gemm(128, 8192, 8192) > 0 and gemm(256, 4096, 8192) > 0
    for M in (128, 130, 255):
        assert size(M, 8192, 8192) == 0 and size(M, 8192, 16384) == gemm(128, 8192, 16384) > 0
    for M in (256, 257, 383):
        assert size(M, 4096, 8192) == gemm(256, 4096, 8192) and size(M, 4096, 8064) == 0
