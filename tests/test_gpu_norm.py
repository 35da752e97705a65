"""GPU tests of the layer / RMS norm: forward, as codes (1x128, dual) and backward, against the formulas in 64 bits.

Tolerances, with u = 2^-24 (half a step of fp32).  A row's sum has at most 32 terms in order in a thread, then 6
levels of lanes and at most 8 waves: fewer than 48 roundings, so
    mean    is off by dm <= 48 u mean|x|
    rstd    relative: the mean square has under 48 + 3 roundings, halved by the root, two more for root and
            reciprocal; the mean's error enters squared: dr <= 30 u + (rstd dm)^2
    y       |g| rstd dm + |g xh| (dr + 3 u) + u (|g xh| + |y|), then half a step of its type.
A column sum over T rows has at most 1 + T / 256 terms in order (a workgroup's rows of one team), then 8 teams, 16
terms of a run of workgroups and 16 runs; each term has 3 roundings: (44 + T / 256) u sum|dy xh|."""
import itertools

import numpy as np
import pytest

from gpu_util import say, torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def half_step(y, dtype):
    """Largest rounding of values y to dtype (an error of half a step, subnormals included)."""
    fi = torch().finfo(dtype)
    return y.abs().clamp_min(fi.tiny) * (fi.eps / 2)


def inputs(T, C, dtype, wdtype, kind, seed, offset=0.25):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    x = (t.randn((T, C), generator=g, device="cuda") + offset).to(dtype)
    w = (1 + 0.3 * t.randn(C, generator=g, device="cuda")).to(wdtype)
    b = (0.2 * t.randn(C, generator=g, device="cuda")).to(wdtype) if kind == 0 else None
    return x, w, b


def reference(x, w, b, eps, kind):
    """(y, mean, rstd) in 64 bits and the bounds of the errors above."""
    x, w = x.double(), w.double()
    A = x.abs().mean(1, keepdim=True)
    mean = x.mean(1, keepdim=True) if kind == 0 else A * 0
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    xh = (x - mean) * rstd
    y = xh * w + (b.double() if b is not None else 0)
    dm = 48 * U * A if kind == 0 else A * 0
    dr = 30 * U + (rstd * dm) ** 2
    dy = w.abs() * rstd * dm + (w * xh).abs() * (dr + 4 * U) + U * y.abs()
    return y, mean[:, 0], rstd[:, 0], dy, dm[:, 0], dr[:, 0]


def near(got, ref, bound, what):
    bad = ((got.double() - ref).abs() > bound) | got.isnan()
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(),
                           float(((got.double() - ref).abs() / bound.clamp_min(1e-300)).max()))


def strided(t, pad):
    """The same values with rows `pad` elements further apart, behind a gap of `pad`."""
    import torch as T
    if not pad:
        return t
    big = T.full((t.shape[0] + 1, t.shape[1] + pad), float("nan"), device=t.device).to(t.dtype) if t.dtype.is_floating_point \
        else T.zeros((t.shape[0] + 1, t.shape[1] + pad), device=t.device, dtype=t.dtype)
    v = big.view(-1)[pad:][: t.shape[0] * (t.shape[1] + pad)].view(t.shape[0], -1)[:, : t.shape[1]]
    v.copy_(t)
    return v


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 63), (2, 64), (33, 512), (4, 520), (1, 1000), (130, 1024), (7, 1032), (1, 2048),
          (67, 2048), (9, 2056), (50, 128), (61, 129), (40, 256), (3, 4096), (2, 4104), (5, 8192), (3, 8200), (2, 16384), (1, 16383), (2100, 136)]


@pytest.mark.parametrize("T,C", SHAPES)
def test_norm_forward(P, T, C):
    t = torch()
    for (dtype, wdtype), kind, pad in itertools.product(
            ((t.bfloat16, t.bfloat16), (t.float32, t.float32), (t.bfloat16, t.float32), (t.float32, t.bfloat16)),
            (P.LAYER_NORM, P.RMS_NORM), (0, 8, 3)):
        say(f"[norm] {T}x{C} {dtype} {wdtype} kind {kind} pad {pad}")
        x, w, b = inputs(T, C, dtype, wdtype, kind, T + C)
        xs = strided(x, pad)
        out = strided(t.zeros_like(x), pad)
        y, mean, rstd = P.puro_layer_norm(xs, w, b, eps=1e-5, kind=kind, y=out)
        ry, rm, rr, by, bm, br = reference(x, w, b, 1e-5, kind)
        near(y, ry, by + half_step(ry, dtype), "y")
        near(rstd, rr, rr * br, "rstd")
        if kind == P.LAYER_NORM:
            near(mean, rm, bm, "mean")
        else:
            assert mean is None


@pytest.mark.parametrize("T,C", [(8200, 2048), (4099, 4096), (2053, 8192), (2051, 16384), (16390, 640), (70001, 128), (33000, 256)])
def test_norm_many_rows(P, T, C):
    """Long inputs, where a team of waves takes several rows in turn: every row as by itself."""
    t = torch()
    for kind in (0, 1):
        say(f"[norm, many rows] {T}x{C} kind {kind}")
        x, w, b = inputs(T, C, t.bfloat16, t.bfloat16, kind, T)
        y, mean, rstd = P.puro_layer_norm(x, w, b, kind=kind)
        q, s = P.puro_layer_norm_quant(x, w, b, kind=kind)
        step = 131072 // max(C, 16)                 # so few rows that a team takes one
        for lo in range(0, T, step):
            part = slice(lo, min(lo + step, T))
            y1, m1, r1 = P.puro_layer_norm(x[part], w, b, kind=kind)
            q1, s1 = P.puro_layer_norm_quant(x[part], w, b, kind=kind)
            assert t.equal(y[part], y1) and t.equal(rstd[part], r1) and (kind == 1 or t.equal(mean[part], m1))
            assert t.equal(q[part], q1) and t.equal(s[:, part], s1)
        ry, rm, rr, by, _, br = reference(x[-40:], w, b, 1e-5, kind)
        near(y[-40:], ry, by + half_step(ry, t.bfloat16), "y")
        near(rstd[-40:], rr, rr * br, "rstd")
        T128 = T // 128 * 128
        d = P.puro_layer_norm_quant_dual(x[:T128], w, b, kind=kind)
        assert t.equal(d[0], q[:T128]) and t.equal(d[1], s[:, :T128]) and t.equal(d[5], rstd[:T128])


def test_norm_leaves_gaps_alone_and_runs_in_place(P):
    t = torch()
    x, w, b = inputs(5, 100, t.bfloat16, t.float32, 0, 3)
    big = t.full((5, 131), 7.0, dtype=t.bfloat16, device="cuda")
    P.puro_layer_norm(x, w, b, y=big[:, 3:103])
    assert (big[:, :3] == 7).all() and (big[:, 103:] == 7).all()
    for C in (100, 2048, 8192):
        x, w, b = inputs(37, C, t.float32, t.float32, 0, 4)
        y, m, r = P.puro_layer_norm(x, w, b)
        z, m2, r2 = P.puro_layer_norm(x, w, b, y=x)
        assert z is x and t.equal(x, y) and t.equal(m, m2) and t.equal(r, r2)


def test_norm_special_rows(P):
    """Rows apart: constant ones, large offsets, infinities and NaN stay in their rows; eps = 0."""
    t = torch()
    for C in (256, 2048, 4096, 12000):
        x, w, b = inputs(6, C, t.float32, t.float32, 0, C)
        clean, _, _ = P.puro_layer_norm(x, w, b)
        x[1] = 3.0
        x[2, C // 2] = float("inf")
        x[3, 5] = float("nan")
        x[4] = x[4] + 1000.0
        y, mean, rstd = P.puro_layer_norm(x, w, b)
        assert t.equal(y[0], clean[0]) and t.equal(y[5], clean[5])
        # a constant row: the mean has 48 roundings, and the difference is divided by sqrt(eps) = 1 / 316.3
        near(y[1], b.double(), w.double().abs() * 3 * 48 * U * 317 + U * b.double().abs(), "constant")
        assert y[2].isnan().any() and y[3].isnan().all() and mean[3].isnan()
        ry, rm, rr, by, bm, br = reference(x[4:5], w, b, 1e-5, 0)
        near(y[4:5], ry, by + half_step(ry, t.float32), "offset")
        z, _, r0 = P.puro_layer_norm(x[:1], w, b, eps=0.0)
        ry, _, rr, by, _, br = reference(x[:1], w, b, 0.0, 0)
        near(z, ry, by + half_step(ry, t.float32), "eps 0")
        zeros, _, _ = P.puro_layer_norm(t.zeros_like(x), w, b)
        assert t.equal(zeros, b.expand_as(x))


def test_norm_empty(P):
    t = torch()
    w = t.ones(64, device="cuda")
    y, m, r = P.puro_layer_norm(t.empty((0, 64), device="cuda"), w)
    assert y.shape == (0, 64) and m.shape == (0,) and r.shape == (0,)
    y, m, r = P.puro_layer_norm(t.empty((3, 0), device="cuda"), t.empty(0, device="cuda"))
    assert y.shape == (3, 0)


def folded(by, x, w, rr, rm):
    """The quantized forms compute (x r - mu r) g + b in two FMAs: besides the bound of y, one rounding of mu r and
    one of the difference, whose terms are |x| r and |mu| r."""
    r, m = rr[:, None], rm[:, None]
    return by + 2 * U * w.double().abs() * r * (m.abs() + (x.double() - m).abs())


def codes_near(P, q, s, y, by, what):
    """Codes q [R, K] and scales s [K/128, R] against the fp64 norm y [R, K] with error bound by.  The scale is the
    group's maximum / 448 (three roundings); a code times its scale is within half an E4M3 step of y (2^-4 of the value,
    2^-10 of the scale where subnormal), the product y r and the reciprocal add 4 u."""
    t = torch()
    R, K = y.shape
    v, d = y.view(R, K // 128, 128), by.view(R, K // 128, 128)
    amax = v.abs().amax(2)
    ref_s = (amax.clamp_min(2.0 ** -96) / 448).t()
    near(s, ref_s, ref_s * 3 * U + (d.amax(2) / 448).t(), what + " scales")
    sc = s.double().t().repeat_interleave(128, 1)
    val = q.view(t.float8_e4m3fn).double() * sc
    eps8 = t.finfo(t.float8_e4m3fn).eps / 2                 # 2^-4
    step = t.maximum((y.abs() + by) * eps8, sc * 2.0 ** -10)
    # (a code of 448 may stand for a value a few roundings above 448 s)
    near(val, y, step * (1 + 2.0 ** -10) + by + 8 * U * y.abs(), what + " codes")


@pytest.mark.parametrize("T,C", [(1, 128), (3, 256), (17, 640), (1, 2048), (70, 2048), (129, 1152), (5, 4096), (2, 8192),
                                 (3, 16384)])
def test_norm_quant_rows(P, T, C):
    t = torch()
    for dtype, kind in itertools.product((t.bfloat16, t.float32), (0, 1)):
        say(f"[norm quant] {T}x{C} {dtype} kind {kind}")
        x, w, b = inputs(T, C, dtype, t.bfloat16, kind, T + C)
        mean = t.empty(T, device="cuda") if kind == 0 else None
        rstd = t.empty(T, device="cuda")
        q, s = P.puro_layer_norm_quant(strided(x, 16), w, b, kind=kind, q=strided(t.zeros((T, C), dtype=t.uint8, device="cuda"), 16),
                                       mean=mean, rstd=rstd)
        y, m, r = P.puro_layer_norm(x, w, b, kind=kind)
        assert t.equal(r, rstd) and (kind == 1 or t.equal(m, mean))
        ry, rm, rr, by, _, _ = reference(x, w, b, 1e-5, kind)
        codes_near(P, q, s, ry, folded(by, x, w, rr, rm), "1x128")


@pytest.mark.parametrize("T,C", [(128, 128), (256, 384), (384, 2048), (128, 4224), (4096, 256), (128, 16384)])
def test_norm_quant_dual(P, T, C):
    t = torch()
    for dtype, kind in itertools.product((t.bfloat16, t.float32), (0, 1)):
        say(f"[norm quant dual] {T}x{C} {dtype} kind {kind}")
        x, w, b = inputs(T, C, dtype, t.float32, kind, T + C)
        q, s, qT, sT, mean, rstd = P.puro_layer_norm_quant_dual(x, w, b, kind=kind)
        q1, s1 = P.puro_layer_norm_quant(x, w, b, kind=kind)
        y, m, r = P.puro_layer_norm(x, w, b, kind=kind)
        assert t.equal(q, q1) and t.equal(s, s1), "the two forms' row codes differ"
        assert t.equal(r, rstd) and (kind == 1 or t.equal(m, mean))
        ry, rm, rr, by, _, _ = reference(x, w, b, 1e-5, kind)
        by = folded(by, x, w, rr, rm)
        codes_near(P, qT, sT, ry.t().contiguous(), by.t().contiguous(), "128x1")


def test_norm_quant_special_groups(P):
    """A zero group gets the floor's scale and zero codes; a row with a NaN gives NaN codes in that row alone, whose
    scales and those of the other rows it does not touch."""
    t = torch()
    x = t.randn((128, 256), device="cuda").bfloat16()
    w = t.ones(256, device="cuda")
    w[128:] = 0
    q, s, qT, sT, _, _ = P.puro_layer_norm_quant_dual(x, w, kind=1)
    assert (q[:, 128:] & 0x7F == 0).all() and t.equal(s[1], t.full_like(s[1], 2.0 ** -96) / 448)
    assert (qT[128:] & 0x7F == 0).all()
    x[3, 7] = float("nan")
    q2, s2 = P.puro_layer_norm_quant(x, w, kind=1)
    assert (q2[3] & 0x7F == 0x7F).all()
    keep = [i for i in range(128) if i != 3]
    assert t.equal(q2[keep], q[keep]) and t.equal(s2[:, keep], s[:, keep])
    q3, s3, qT3, sT3, _, _ = P.puro_layer_norm_quant_dual(x, w, kind=1)
    assert t.equal(q3, q2) and t.equal(s3, s2) and (qT3[:, 3] & 0x7F == 0x7F).all() and sT3.isfinite().all()
    x[3, 7] = x[3, 8]
    x[:, 9] = 0
    rest = P.puro_layer_norm_quant_dual(x, w, kind=1)
    x[3, 9] = float("nan")
    bad = P.puro_layer_norm_quant_dual(x, w, kind=1)
    assert (bad[2][:, keep] == rest[2][:, keep]).float().mean() > 0.9    # a column's maximum may have been row 3's


def ref_backward(dy, x, w, mean, rstd, kind):
    x, dy, w = x.double(), dy.double(), w.double()
    m = mean.double()[:, None] if kind == 0 else 0.0
    r = rstd.double()[:, None]
    C, T = x.shape[1], x.shape[0]
    xh = (x - m) * r
    g = dy * w
    c1 = g.mean(1, keepdim=True) if kind == 0 else 0 * r
    c2 = (g * xh).mean(1, keepdim=True)
    dx = r * (g - c1 - xh * c2)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    # row sums: under 48 roundings, terms of at most 4; the combination four more
    bx = U * r * (6 * g.abs() + 54 * a1 * (1 if kind == 0 else 0) + 58 * xh.abs() * a2 + 6 * (xh * c2).abs() + 3 * abs(c1))
    n = 44 + T / 256
    return dx, (dy * xh).sum(0), dy.sum(0), bx, n * U * (dy * xh).abs().sum(0), n * U * dy.abs().sum(0)


@pytest.mark.parametrize("T,C", [(1, 1), (1, 8), (2, 7), (17, 100), (90, 128), (200, 200), (16, 512), (65, 512), (300, 1000), (1027, 1000), (40, 2048),
                                 (513, 2048), (5, 4096), (33, 4100), (9, 8192), (1, 16384), (19, 16376), (4500, 256), (6001, 2048), (2100, 4096), (1300, 8192), (40000, 120)])
def test_norm_backward(P, T, C):
    t = torch()
    for (dtype, wdtype), kind, pad in itertools.product(((t.bfloat16, t.bfloat16), (t.float32, t.float32), (t.bfloat16, t.float32)),
                                                        (0, 1), (0, 8, 5)):
        say(f"[norm backward] {T}x{C} {dtype} {wdtype} kind {kind} pad {pad}")
        x, w, b = inputs(T, C, dtype, wdtype, kind, T + C)
        dy = (t.randn_like(x.float()) * 1e-2).to(dtype)
        _, mean, rstd = P.puro_layer_norm(x, w, b, kind=kind)
        out = strided(t.zeros_like(x), pad)
        dx, dw, db = P.puro_layer_norm_backward(strided(dy, pad), strided(x, pad), w, mean, rstd, kind=kind, dx=out)
        rx, rw, rb, bx, bw, bb = ref_backward(dy, x, w, mean, rstd, kind)
        near(dx, rx, bx + half_step(rx, dtype), "dx")
        near(dw, rw, bw + 1e-40, "dweight")
        near(db, rb, bb + 1e-40, "dbias")
        # adding to gradients that are there: one fp32 addition per element
        w0, b0 = t.randn(C, device="cuda"), t.randn(C, device="cuda")
        w1, b1 = w0.clone(), b0.clone()
        P.puro_layer_norm_backward(dy, x, w, mean, rstd, kind=kind, dweight=w1, dbias=b1, accumulate=True)
        dx2, dw2, db2 = P.puro_layer_norm_backward(dy, x, w, mean, rstd, kind=kind)
        assert t.equal(w1, w0 + dw2) and t.equal(b1, b0 + db2)
        dx3, dw3, none = P.puro_layer_norm_backward(dy, x, w, mean, rstd, kind=kind, with_bias=False)
        assert none is None and t.equal(dw3, dw2) and t.equal(dx3, dx2)
        # in place over dy
        dyc = dy.clone()
        P.puro_layer_norm_backward(dyc, x, w, mean, rstd, kind=kind, dx=dyc)
        assert t.equal(dyc, dx2)


def test_norm_backward_against_differences(P):
    """The derivative of sum(dy y) along random directions, by central differences of the 64-bit formula: the
    step h = 1e-5 leaves h^2 and 64-bit roundings / h, both below 1e-8 of the terms' sum."""
    t = torch()
    for kind in (0, 1):
        x, w, b = inputs(9, 200, t.float32, t.float32, kind, 11)
        dy = t.randn_like(x)
        _, mean, rstd = P.puro_layer_norm(x, w, b, kind=kind)
        dx, dw, db = P.puro_layer_norm_backward(dy, x, w, mean, rstd, kind=kind)
        f = lambda x, w, b: (reference(x, w, b, 1e-5, kind)[0] * dy.double())
        X, W = x.double(), w.double()
        B = b.double() if b is not None else t.zeros_like(W)
        h = 1e-5
        for which, grad in ((0, dx), (1, dw), (2, db)):
            d = [t.zeros_like(X), t.zeros_like(W), t.zeros_like(B)]
            d[which] = t.randn_like(d[which])
            plus = f(X + h * d[0], W + h * d[1], B + h * d[2])
            minus = f(X - h * d[0], W - h * d[1], B - h * d[2])
            diff = float(((plus - minus).sum()) / (2 * h))
            got = float((grad.double() * d[which]).sum())
            size = float((grad.double() * d[which]).abs().sum()) + float(plus.abs().sum())
            assert abs(diff - got) <= (100 * U + 1e-7) * size, (kind, which, diff, got)


def test_norm_backward_empty_and_constant_rows(P):
    t = torch()
    w = t.ones(40, device="cuda")
    e = t.empty((0, 40), device="cuda")
    s = t.empty(0, device="cuda")
    dw, db = t.ones(40, device="cuda"), t.ones(40, device="cuda")
    P.puro_layer_norm_backward(e, e, w, s, s, dweight=dw, dbias=db, accumulate=True)
    assert (dw == 1).all() and (db == 1).all()
    P.puro_layer_norm_backward(e, e, w, s, s, dweight=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()
    x = t.full((4, 40), 2.0, device="cuda")
    _, m, r = P.puro_layer_norm(x, w)
    dx, dw, db = P.puro_layer_norm_backward(t.ones_like(x), x, w, m, r)
    assert dx.isfinite().all() and t.equal(db, t.full_like(db, 4.0))


def test_norm_on_another_stream_and_in_a_graph(P):
    t = torch()
    x, w, b = inputs(300, 2048, t.bfloat16, t.bfloat16, 0, 5)
    dy = t.randn_like(x)
    y, m, r = P.puro_layer_norm(x, w, b)
    dx, dw, db = P.puro_layer_norm_backward(dy, x, w, m, r)
    q, s = P.puro_layer_norm_quant(x, w, b)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    y2, m2, r2 = P.puro_layer_norm(x, w, b, stream=side)
    dx2, dw2, db2 = P.puro_layer_norm_backward(dy, x, w, m2, r2, stream=side.cuda_stream)
    q2, s2 = P.puro_layer_norm_quant(x, w, b, stream=side)
    t.cuda.synchronize()
    for a, c in ((y, y2), (m, m2), (r, r2), (dx, dx2), (dw, dw2), (db, db2), (q, q2), (s, s2)):
        assert t.equal(a, c)
    graph = t.cuda.CUDAGraph()
    xin, dyin = x.clone(), dy.clone()
    with t.cuda.graph(graph):
        gy, gm, gr = P.puro_layer_norm(xin, w, b)
        gdx, gdw, gdb = P.puro_layer_norm_backward(dyin, xin, w, gm, gr)
        gq = P.puro_layer_norm_quant(xin, w, b)
    for k in range(3):
        xin.copy_(x * (k + 1))
        dyin.copy_(dy / (k + 1))
        graph.replay()
        t.cuda.synchronize()
        ey, em, er = P.puro_layer_norm(xin, w, b)
        edx, edw, edb = P.puro_layer_norm_backward(dyin, xin, w, em, er)
        eq = P.puro_layer_norm_quant(xin, w, b)
        for a, c in ((gy, ey), (gm, em), (gr, er), (gdx, edx), (gdw, edw), (gdb, edb), (gq[0], eq[0]), (gq[1], eq[1])):
            assert t.equal(a, c), k


def test_two_streams_at_once(P):
    """Calls on two streams that are not ordered, each with outputs and a workspace of its own."""
    t = torch()
    work = []
    for k in range(2):
        x, w, b = inputs(2000, 2048, t.bfloat16, t.bfloat16, 0, k)
        dy = t.randn_like(x)
        y, m, r = P.puro_layer_norm(x, w, b)
        work.append((x, w, b, dy, m, r, y, P.puro_layer_norm_backward(dy, x, w, m, r)))
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    t.cuda.synchronize()
    got = []
    for n in range(10):
        for s, (x, w, b, dy, m, r, y, want) in zip(streams, work):
            got.append((P.puro_layer_norm(x, w, b, stream=s)[0], y))
            got += list(zip(P.puro_layer_norm_backward(dy, x, w, m, r, stream=s), want))
    t.cuda.synchronize()
    for a, c in got:
        assert t.equal(a, c)


def test_norm_binding_refusals(P):
    t = torch()
    x, w, b = inputs(4, 128, t.bfloat16, t.bfloat16, 0, 1)
    with pytest.raises(TypeError):
        P.puro_layer_norm(x, w, b.float())
    with pytest.raises(ValueError):
        P.puro_layer_norm(x, w[:64])
    with pytest.raises(ValueError):
        P.puro_layer_norm(x.t(), w)
    with pytest.raises(ValueError):
        P.puro_layer_norm(x, w, kind=5)
    with pytest.raises(ValueError):
        P.puro_layer_norm(x, w, kind=P.RMS_NORM, mean=t.empty(4, device="cuda"))
    with pytest.raises(P.PuroError):
        P.puro_layer_norm(x, w, eps=-1.0)
    with pytest.raises(P.PuroError):
        P.puro_layer_norm_quant(x[:, :100], w[:100])
    with pytest.raises(P.PuroError):
        P.puro_layer_norm_quant_dual(x, w)                        # 4 rows
    with pytest.raises(ValueError):
        P.puro_layer_norm(x[:1].expand(4, 128), w, y=x[:1].expand(4, 128))
    with pytest.raises(TypeError):
        P.puro_layer_norm_backward(x, x, w, None, t.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        P.puro_layer_norm_backward(x, x, w, t.ones(4, device="cuda"), t.ones(4, device="cuda"), accumulate=True)


def test_norm_past_32_bit_offsets(P):
    """A strided view whose rows lie more than 2^31 elements apart (read and written)."""
    t = torch()
    ld = (1 << 31) + 64
    big = t.empty(2 * ld, dtype=t.bfloat16, device="cuda")
    x = big.as_strided((2, 256), (ld, 1))
    v, w, b = inputs(2, 256, t.bfloat16, t.bfloat16, 0, 9)
    x.copy_(v)
    ry = P.puro_layer_norm(v, w, b)
    y = big.as_strided((2, 256), (ld, 1), 512)
    P.puro_layer_norm(x, w, b, y=y)
    assert t.equal(y, ry[0])
    dx, dw, db = P.puro_layer_norm_backward(v, v, w, ry[1], ry[2])
    dx2, dw2, db2 = P.puro_layer_norm_backward(x, x, w, ry[1], ry[2], dx=y)
    assert t.equal(dx, y) and t.equal(dw, dw2) and t.equal(db, db2)
    q, s = P.puro_layer_norm_quant(x, w, b)
    q2, s2 = P.puro_layer_norm_quant(v, w, b)
    assert t.equal(q, q2) and t.equal(s, s2)


def test_norm_past_32_bit_elements(P):
    """More than 2^31 elements: the last rows, and the last token block of every column, as by themselves."""
    t = torch()
    T, C = 262272, 8192
    assert T * C > 2 ** 31
    g = t.Generator(device="cuda")
    g.manual_seed(1)
    x = t.randn((T, C), generator=g, device="cuda", dtype=t.bfloat16)
    w, b = t.randn(C, device="cuda"), t.randn(C, device="cuda")
    tail = slice(T - 128, T)
    say(f"[norm, large] {T}x{C}")
    y, m, r = P.puro_layer_norm(x, w, b)
    y1, m1, r1 = P.puro_layer_norm(x[tail], w, b)
    assert t.equal(y[tail], y1) and t.equal(m[tail], m1) and t.equal(r[tail], r1)
    dx, dw, db = P.puro_layer_norm_backward(y, x, w, m, r)
    dx1, _, _ = P.puro_layer_norm_backward(y1, x[tail], w, m1, r1)
    assert t.equal(dx[tail], dx1) and dw.isfinite().all() and db.isfinite().all()
    del dx, y
    q, s, qT, sT, _, _ = P.puro_layer_norm_quant_dual(x, w, b)
    q1, s1, qT1, sT1, _, _ = P.puro_layer_norm_quant_dual(x[tail], w, b)
    assert t.equal(q[tail], q1) and t.equal(s[:, tail], s1)
    assert t.equal(qT[:, tail], qT1) and t.equal(sT[-1:], sT1)
    del q, qT
    q, s = P.puro_layer_norm_quant(x, w, b)
    assert t.equal(q[tail], q1) and t.equal(s[:, tail], s1)


def test_more_short_rows_than_a_launch_has_threads(P):
    """2^30 rows and some: an RMS norm of single elements is their sign, but for eps (0: exactly one rounding of |x|'s
    reciprocal root, 2^-8 in bf16); the rows at the end as by themselves."""
    t = torch()
    T = (1 << 30) + 77
    x = t.ones((T, 1), device="cuda", dtype=t.bfloat16)
    x[::3] = -2
    w = t.ones(1, device="cuda", dtype=t.bfloat16)
    say(f"[norm, long] {T}x1")
    y, _, r = P.puro_layer_norm(x, w, eps=0.0, kind=P.RMS_NORM)
    assert float((y.abs() - 1).abs().max()) <= 2.0 ** -8 and t.equal(y < 0, x < 0)
    tail = x[-1000:].contiguous()
    y1, _, r1 = P.puro_layer_norm(tail, w, eps=0.0, kind=P.RMS_NORM)
    assert t.equal(y[-1000:], y1) and t.equal(r[-1000:], r1)
