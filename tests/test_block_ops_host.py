"""Host-side checks of the residual sum with its norms, the rotary positions and the AdamW step (no GPU, no kernel launched):
every call below has an invalid argument or an empty shape, so the library returns before any HIP call."""
import ctypes
import math
import os
import re

import pytest

import blockwise_scaled_fp8_quant_amd as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULLPTR, SHAPE, ALIGN, LD, MODE, DTYPE, WORKSPACE, UNSUP, ARG = 0, -1, -2, -3, -4, -5, -6, -7, -9, -10
A = [0x100000 * (i + 1) for i in range(16)]       # never dereferenced: validation fails first
MIS = A[0] + 8
BF16, FP32 = 0, 1


def test_structs_are_the_header_s():
    """The fields of each ctypes structure are the header's, in its order."""
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "puro_ops.h")).read(), flags=re.S)
    for struct, name in ((P.Residual, "puro_residual"), (P.ResidualGrad, "puro_residual_grad"), (P.AdamwJob, "puro_adamw_job"),
                         (P.AdamwHyper, "puro_adamw_hyper")):
        body = re.search(r"typedef struct " + name + r" \{(.*?)\} " + name + ";", src, flags=re.S).group(1)
        kinds = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "uint64_t": ctypes.c_uint64, "float": ctypes.c_float,
                 "double": ctypes.c_double}
        want = []
        for line in body.split(";"):
            m = re.match(r"\s*(?:const )?(\w+)\s*(\*?)\s*(.+)", line.strip(), flags=re.S)
            if m:
                for field in m.group(3).split(","):
                    pointer = m.group(2) or field.strip().startswith("*")
                    want.append((field.strip(" *\n"), ctypes.c_void_p if pointer else kinds[m.group(1)]))
        assert [(n, k) for n, k in struct._fields_] == want


def struct(of, base, **k):
    return of(**{**base, **k})


RES = dict(kind=0, x_dtype=BF16, w_dtype=BF16, T=4, C=256, h=A[0], ldh=256, x=A[1], ldx=256, weight=A[2], bias=A[3], gate=A[4],
           post_weight=A[5], scale=0.5, eps=1e-5, h_out=A[6], ldh_out=256, mean=A[7], rstd=A[8], post_mean=A[9], post_rstd=A[10])


def residual(y=A[11], ldy=256, **k):
    return P.lib.puro_residual_norm(ctypes.byref(struct(P.Residual, RES, **k)), y, ldy, None)


def quant(q=A[11], ldq=256, s=A[12], **k):
    return P.lib.puro_residual_norm_quant(ctypes.byref(struct(P.Residual, RES, **k)), q, ldq, s, None)


def dual(q=A[11], ldq=256, s=A[12], qT=A[13], ldqT=256, sT=A[14], **k):
    return P.lib.puro_residual_norm_quant_dual(ctypes.byref(struct(P.Residual, {**RES, "T": 256}, **k)), q, ldq, s, qT, ldqT, sT, None)


def test_residual_refusals():
    assert P.lib.puro_residual_norm(None, A[11], 256, None) == NULLPTR
    assert residual(T=0) == OK and residual(C=0) == OK and residual(T=0, h=None, x=None, y=None) == OK
    assert residual(kind=2) == MODE and residual(x_dtype=2) == DTYPE and residual(w_dtype=-1) == DTYPE
    assert residual(T=-1) == SHAPE and residual(C=-1) == SHAPE
    for v in (-1e-5, math.nan, math.inf):
        assert residual(eps=v) == ARG
    for v in (math.nan, math.inf, -math.inf):
        assert residual(scale=v) == ARG
    assert residual(kind=1) == ARG and residual(kind=1, mean=None) == ARG                # an RMS norm has no means
    assert residual(post_weight=None) == ARG and residual(post_weight=None, post_mean=None) == ARG
    for name in ("h", "x", "weight", "h_out"):
        assert residual(**{name: None}) == NULLPTR, name
        assert residual(**{name: A[0] + 1}) == ALIGN, name
    assert residual(y=None) == NULLPTR and residual(y=A[11] + 1) == ALIGN and residual(y=A[6]) == ARG
    for name in ("gate", "post_weight", "bias"):
        assert residual(**{name: A[0] + 1}) == ALIGN, name
    for name in ("mean", "rstd", "post_mean", "post_rstd"):
        assert residual(**{name: A[0] + 2}) == ALIGN, name
    for name in ("ldh", "ldx", "ldh_out"):
        assert residual(**{name: 255}) == LD, name
    assert residual(ldy=255) == LD
    wide = dict(C=16385, ldh=16385, ldx=16385, ldh_out=16385)
    assert residual(**wide, ldy=16385) == UNSUP


def test_residual_codes_refusals():
    assert quant(T=0) == OK and quant(C=0) == OK and quant(C=200) == SHAPE and dual(C=200) == SHAPE and dual(T=100) == SHAPE
    assert P.lib.puro_residual_norm_quant(None, A[0], 256, A[1], None) == NULLPTR
    assert P.lib.puro_residual_norm_quant_dual(None, A[0], 256, A[1], A[2], 256, A[3], None) == NULLPTR
    for call in (quant, dual):
        for name in ("h", "x", "h_out", "weight", "q", "s"):
            assert call(**{name: None}) == NULLPTR, name
            assert call(**{name: MIS}) == ALIGN, name
        for name in ("gate", "post_weight", "bias"):
            assert call(**{name: MIS}) == ALIGN, name
        for name in ("ldh", "ldx", "ldh_out"):
            assert call(**{name: 260}) == LD and call(**{name: 128}) == LD, name
        assert call(ldq=264) == LD and call(ldq=128) == LD and call(scale=math.nan) == ARG
    assert dual(qT=None) == NULLPTR and dual(sT=MIS) == ALIGN and dual(rstd=None) == NULLPTR and dual(mean=None) == NULLPTR
    assert dual(ldqT=128) == LD and dual(ldqT=264) == LD


GRAD = dict(kind=0, x_dtype=BF16, w_dtype=BF16, T=64, C=256, dy=A[0], lddy=256, h_out=A[1], ldh_out=256, dh_out=A[2], lddh_out=256,
            x=A[3], ldx=256, weight=A[4], gate=A[5], post_weight=A[6], scale=0.5, mean=A[7], rstd=A[8], post_mean=A[9],
            post_rstd=A[10], dh=A[11], lddh=256, dx=A[12], lddx=256, dweight=A[13], dbias=A[13] + 4096, dgate=A[14],
            dpost_weight=A[15], accumulate=0)


def back(ws=A[0], wb=1 << 30, **k):
    return P.lib.puro_residual_norm_backward(ctypes.byref(struct(P.ResidualGrad, GRAD, **k)), ws, wb, None)


def test_residual_backward_refusals():
    assert P.lib.puro_residual_norm_backward(None, A[0], 1 << 30, None) == NULLPTR
    assert back(C=0) == OK and back(T=0, accumulate=1) == OK
    assert back(kind=3) == MODE and back(x_dtype=7) == DTYPE and back(T=-1) == SHAPE and back(accumulate=2) == ARG
    assert back(kind=1) == ARG and back(kind=1, mean=None) == ARG and back(scale=math.inf) == ARG
    assert back(post_weight=None) == ARG and back(gate=None) == ARG
    for name in ("dy", "h_out", "x", "weight", "mean", "rstd", "post_mean", "post_rstd", "dh", "dx", "dweight"):
        assert back(**{name: None}) == NULLPTR, name
    for name in ("dy", "h_out", "dh_out", "x", "dh", "dx", "weight", "gate", "post_weight"):
        assert back(**{name: A[0] + 1}) == ALIGN, name
    for name in ("mean", "rstd", "post_mean", "post_rstd", "dweight", "dbias", "dgate", "dpost_weight"):
        assert back(**{name: A[0] + 2}) == ALIGN, name
    for name in ("lddy", "ldh_out", "lddh_out", "ldx", "lddh", "lddx"):
        assert back(**{name: 255}) == LD, name
    assert back(dx=A[11]) == ARG and back(C=16385) == UNSUP
    size = P.puro_residual_norm_backward_workspace_size
    big = {k: 2048 for k in ("C", "lddy", "ldh_out", "lddh_out", "ldx", "lddh", "lddx")}
    need = size(16384, 2048, True)
    assert need > size(16384, 2048, False) > 0
    assert back(T=16384, **big, wb=need - 1) == WORKSPACE and back(T=16384, **big, ws=None) == WORKSPACE
    assert back(T=16384, **big, ws=MIS) == ALIGN
    for gated in (False, True):
        assert size(0, 2048, gated) == size(1, 2048, gated) == size(8, 1 << 20, gated) == 0


def test_residual_backward_workgroups_grow_with_the_rows():
    """No team takes more than 64 times 64 rows, and no more than 64 where the kernel adds no runs (more than 8192
    columns, with a gate or norm more than 4096); a launch has fewer than 2^32 threads."""
    for C, lanes in ((8, 16), (128, 16), (200, 32), (1000, 64), (2000, 128), (4096, 256), (4104, 512), (8200, 512), (16384, 512)):
        for gated in (False, True):
            most = 64 if C > (4096 if gated else 8192) else 4096
            for T in (1000, 16384, 262145, 1 << 20, (1 << 20) + 1, 10 ** 7):
                blocks = max(P.puro_residual_norm_backward_workspace_size(T, C, gated) // (4 * (3 if gated else 2) * C), 1)
                assert blocks * (512 // lanes) * most >= T and blocks * 512 < 1 << 32
                assert blocks <= 256 or T > 256 * most


def rotary(xd=BF16, layout=0, inverse=0, x=A[0], ld_t=512, ld_h=128, T=4, H=4, D=128, pos=A[1], start=0, freqs=A[2], pairs=64, scale=1.0,
           y=A[3], ldy_t=512, ldy_h=128):
    return P.lib.puro_rotary(xd, layout, inverse, x, ld_t, ld_h, T, H, D, pos, start, freqs, pairs, scale, y, ldy_t, ldy_h, None)


def test_rotary_refusals():
    assert rotary(T=0) == OK and rotary(H=0) == OK and rotary(D=0, pairs=0) == OK
    assert rotary(layout=2) == MODE and rotary(xd=2) == DTYPE and rotary(inverse=2) == ARG
    assert rotary(T=-1) == SHAPE and rotary(H=-1) == SHAPE and rotary(D=-1) == SHAPE and rotary(pairs=65) == SHAPE and rotary(pairs=-1) == SHAPE
    assert rotary(scale=math.nan) == ARG and rotary(scale=math.inf) == ARG
    assert rotary(x=None) == NULLPTR and rotary(y=None) == NULLPTR and rotary(freqs=None) == NULLPTR
    assert rotary(x=A[0] + 1) == ALIGN and rotary(xd=FP32, y=A[3] + 2) == ALIGN and rotary(freqs=A[2] + 4) == ALIGN and rotary(pos=A[1] + 4) == ALIGN
    assert rotary(ld_t=-1) == LD and rotary(ldy_h=127) == LD and rotary(ldy_t=511) == LD and rotary(ldy_t=0) == LD
    assert rotary(ldy_t=128, ldy_h=511) == LD                             # heads outermost, and one short of four tokens
    assert rotary(T=1 << 31, ldy_t=1 << 40, ldy_h=1 << 62) == LD          # (the product does not wrap)
    assert rotary(y=A[0], ldy_t=1024) == ARG and rotary(y=A[0], ldy_t=128, ldy_h=512) == ARG
    assert rotary(T=1 << 31) == UNSUP and rotary(H=1 << 31, ldy_t=1 << 40) == UNSUP
    assert rotary(D=(1 << 30) + 1, ldy_h=1 << 31, ldy_t=1 << 40) == UNSUP
    assert rotary(D=8192, pairs=2049, ldy_h=8192, ldy_t=1 << 20) == UNSUP


JOB = dict(param=A[0], master=None, grad=A[1], exp_avg=A[2], exp_avg_sq=A[3], avg_scale=None, sq_scale=None, n=300, param_dtype=FP32,
           grad_dtype=FP32)
JOB8 = {**JOB, "avg_scale": A[4], "sq_scale": A[5]}
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1, max_norm=1.0)


def adamw(*jobs, n=None, **h):
    arr = (P.AdamwJob * max(1, len(jobs)))(*[P.AdamwJob(**j) for j in jobs])
    return P.lib.puro_adamw(arr, len(jobs) if n is None else n, ctypes.byref(P.AdamwHyper(**{**HYPER, **h})), None)


def test_adamw_refusals():
    assert adamw() == OK and adamw({**JOB, "n": 0, "param": None}) == OK and adamw(n=-1) == SHAPE
    assert P.lib.puro_adamw(None, 1, ctypes.byref(P.AdamwHyper(**HYPER)), None) == NULLPTR
    assert P.lib.puro_adamw(None, 0, None, None) == NULLPTR
    for bad in (dict(lr=math.nan), dict(lr=math.inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=math.nan),
                dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan), dict(weight_decay=math.nan), dict(step=0), dict(step=-3),
                dict(norm=A[9], max_norm=-1.0), dict(norm=A[9], max_norm=math.nan)):
        assert adamw(JOB, **bad) == ARG, bad
    assert adamw(norm=A[9] + 2) == ALIGN and adamw(lr_dev=A[9] + 2) == ALIGN and adamw(step_dev=A[9] + 4) == ALIGN
    assert adamw(step_dev=A[9], step=0) == OK
    for base in (JOB, JOB8):
        for name in ("param", "grad", "exp_avg", "exp_avg_sq"):
            assert adamw({**base, name: None}) == NULLPTR, name
        assert adamw({**base, "param": A[0] + 2}) == ALIGN and adamw({**base, "grad": A[1] + 2}) == ALIGN
        assert adamw({**base, "n": -1}) == SHAPE and adamw({**base, "param_dtype": 2}) == DTYPE and adamw({**base, "grad_dtype": 5}) == DTYPE
        assert adamw({**base, "master": A[6]}) == ARG and adamw({**base, "param_dtype": BF16, "master": A[6] + 2}) == ALIGN
    assert adamw({**JOB, "exp_avg": A[2] + 2}) == ALIGN and adamw({**JOB8, "avg_scale": A[4] + 2}) == ALIGN
    assert adamw({**JOB8, "sq_scale": None}) == ARG and adamw({**JOB8, "avg_scale": None}) == ARG
    assert adamw({**JOB, "n": (1 << 42) + 1}) == UNSUP


def test_adamw_refuses_overlaps():
    """300 elements: 1200 bytes in fp32, 300 of codes, 12 of scales."""
    for name, other, last in (("grad", "param", 1196), ("exp_avg", "param", 1196), ("exp_avg_sq", "exp_avg", 1196), ("grad", "exp_avg_sq", 1196)):
        for at in (0, 4, last):
            assert adamw({**JOB, name: JOB[other] + at}) == ARG, (name, other, at)
    for name, other, last in (("exp_avg_sq", "exp_avg", 299), ("avg_scale", "exp_avg", 296), ("sq_scale", "avg_scale", 8)):
        assert adamw({**JOB8, name: JOB8[other] + last}) == ARG, (name, other)
    bf16 = {**JOB8, "param_dtype": BF16, "master": A[6]}
    assert adamw({**bf16, "master": A[0] + 596}) == ARG and adamw({**bf16, "master": A[1]}) == ARG
    second = {**JOB, **{k: JOB[k] + 4096 for k in ("param", "grad", "exp_avg", "exp_avg_sq")}}
    for name in ("param", "exp_avg", "exp_avg_sq"):
        assert adamw(JOB, {**second, name: JOB[name] + 1196}) == ARG
    assert adamw(JOB, {**second, "grad": JOB["param"]}) == ARG
    for name in ("norm", "lr_dev"):
        assert adamw(JOB, **{name: A[0] + 1196}) == ARG and adamw(JOB, **{name: A[2]}) == ARG
    assert adamw(JOB, step_dev=A[3] + 1192) == ARG
    # a gradient may be shared, and side by side is fine: these calls get as far as the next job's mistake
    broken = {**JOB, "n": -1}
    assert adamw(JOB, {**second, "grad": JOB["grad"]}, broken) == SHAPE


def test_binding_refuses_what_the_library_cannot_see():
    import torch
    x, w = torch.zeros(4, 128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        P.puro_residual_norm(x, x, w)                                    # host tensors
    with pytest.raises(TypeError):
        P.puro_residual_norm(x.half(), x, w)
    with pytest.raises(ValueError):
        P.puro_residual_norm(x[0], x, w)
    with pytest.raises(TypeError):
        P.puro_residual_norm(x, x, w, scale="1")
    with pytest.raises(ValueError):
        P.puro_residual_norm_backward(x, x, w, None, w)
    with pytest.raises(ValueError):
        P.puro_rotary(x, w)
    with pytest.raises(TypeError):
        P.puro_rotary(x.half()[None], w)
    with pytest.raises(ValueError):
        P.puro_adamw([w], [w], [w], [w], 1, 1e-3)
    with pytest.raises(TypeError):
        P.puro_adamw([w.half()], [w], [w], [w], 1, 1e-3)
    with pytest.raises(ValueError):
        P.puro_adamw([w], [w, w], [w], [w], 1, 1e-3)


def test_rotary_frequencies():
    """Plain ones by their formula; the scaled ones' ends: the fastest pair is left, the slowest `factor` times slower."""
    from blockwise_scaled_fp8_quant_amd.rotary import rotary_frequencies
    plain, one = rotary_frequencies(64, 5000.0)
    assert one == 1.0 and plain.shape == (32,) and str(plain.dtype) == "torch.float64"
    for i in (0, 7, 31):
        assert math.isclose(float(plain[i]), 5000.0 ** (-2 * i / 64), rel_tol=1e-14)
    linear, one = rotary_frequencies(64, 5000.0, "linear", 4.0)
    assert one == 1.0 and ((linear * 4 - plain).abs() <= 1e-15 * plain).all()
    based, one = rotary_frequencies(64, 5000.0, "base", 4.0)
    assert one == 1.0 and float(based[0]) == 1.0 and math.isclose(float(plain[31] / based[31]), 4.0, rel_tol=1e-12)
    yarn, scale = rotary_frequencies(64, 5000.0, "yarn", 4.0, trained_length=2048)
    turns = 2048 * plain / (2 * math.pi)
    assert math.isclose(scale, 0.1 * math.log(4) + 1)
    for i in range(32):
        kept = min(1.0, max(0.0, (float(turns[i]) - 1) / 31))
        assert math.isclose(float(yarn[i]), float(plain[i]) * (kept + (1 - kept) / 4), rel_tol=1e-12)
    assert float(yarn[0]) == 1.0 and math.isclose(float(yarn[31]) * 4, float(plain[31]), rel_tol=1e-12)
    assert rotary_frequencies(64, 5000.0, "yarn", 1.0, trained_length=2048)[1] == 1.0
    for bad in (dict(columns=7), dict(columns=-2), dict(columns=8, scaling="other"), dict(columns=8, scaling="yarn", factor=2.0),
                dict(columns=8, scaling="yarn", trained_length=9, low=3.0, high=3.0), dict(columns=8, base=0.0),
                dict(columns=8, factor=-1.0), dict(columns=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            rotary_frequencies(**bad)


def test_captured_steps_are_checked(monkeypatch):
    """Every differentiable call made while a graph is recorded is checked before its forward pass starts, with every leaf."""
    import torch
    from blockwise_scaled_fp8_quant_amd import linear, residual, rotary

    class Stop(Exception):
        pass

    def check(leaves):
        raise Stop(sum(isinstance(v, torch.Tensor) for v in leaves))
    monkeypatch.setattr(linear, "check_capture", check)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)

    class OnGpu(torch.Tensor):
        is_cuda = True
    x = torch.zeros((128, 128), dtype=torch.bfloat16).as_subclass(OnGpu)
    full = dict(gate=1.0, post_norm=True)
    freqs, _ = rotary.rotary_frequencies(32)
    for call, tensors in ((lambda: residual.ResidualNorm(128, **full)(x, x), 6),
                          (lambda: residual.Fp8ResidualNormLinear(128, 128, **full)(x, x), 7),
                          (lambda: residual.residual_norm(x, x, x[0]), 3), (lambda: rotary.rotary(x.view(64, 4, 64), freqs), 2),
                          (lambda: rotary.Rotary(32)(x.view(64, 4, 64)), 2)):
        with pytest.raises(Stop) as stopped:
            call()
        assert stopped.value.args == (tensors,)
