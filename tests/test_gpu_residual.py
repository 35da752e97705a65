"""GPU tests of the residual sum with its norms: forward (as a tensor, as codes, as codes of both orientations) and backward,
against the formulas in 64 bits.

The norm of the sum is held to the norm's own entry points, which have their tests: y, codes, scales and statistics are those
of h_out as written, bit for bit.  What is left is h_out and the statistics of the norm behind the block.  Tolerances, with
u = 2^-24 (half a step of fp32), and the norm's bounds of tests/test_gpu_norm.py (a row's sum has fewer than 48 roundings):
    p       x, or the norm's bound of norm(x) post_weight
    h_out   the factor scale gate post_weight has three roundings (scale from 64 bits, two products), the sum one:
            |scale gate| dp + 4 u |scale gate p| + u |h_out|, then half a step of its type
    D       the norm's backward bound, the product with rstd and the sum with dh_out: + 2 u |dh_out| + u |D|
    dx      f = scale gate (post_weight): without a norm |f| dD + 4 u |f D|; with one, the error of f D (|f| dD + 4 u |f D|)
            goes through the norm's backward pass, rstd (|e| + mean|e| + |xh| mean|e xh|), and its own bound is added
    sums    a column's sum over T rows has at most 1 + T / 256 terms in order, then 8 teams, 16 terms of a run of workgroups
            and 16 runs; each term has 3 roundings, the vector behind the sum 3: n = 47 + T / 256, n u sum|term|, and the
            terms' own error, sum |q| dD."""
import itertools

import pytest

from gpu_util import say, torch
from test_gpu_norm import half_step, near, reference, strided

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def inputs(T, C, dtype, wdtype, kind, gate, post, seed):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: t.randn(s, generator=g, device="cuda")
    h, x = (2 * r(T, C)).to(dtype), (r(T, C) + 0.25).to(dtype)
    vec = {"weight": (1 + 0.3 * r(C)).to(wdtype), "bias": (0.2 * r(C)).to(wdtype) if kind == 0 else None,
           "gate": (0.4 + 0.3 * r(C)).to(wdtype) if gate else None, "post_weight": (1 + 0.2 * r(C)).to(wdtype) if post else None}
    return h, x, vec


def one(v):
    return 1.0 if v is None else v.double()


def sum_reference(h, x, vec, scale, kind):
    """(h_out, its bound without the final rounding, post_mean, post_rstd, their bounds) in 64 bits."""
    f = scale * one(vec["gate"])
    if vec["post_weight"] is None:
        p, dp, stats = x.double(), 0.0, None
    else:
        p, pm, pr, dp, dm, dr = reference(x, vec["post_weight"], None, EPS, kind)
        stats = (pm, pr, dm, dr)
    total = h.double() + f * p
    f = abs(f)
    return total, f * dp + 4 * U * (f * p.abs()) + U * total.abs(), stats


SHAPES = [(1, 1), (3, 7), (5, 63), (2, 64), (33, 512), (4, 520), (1, 1000), (130, 1024), (1, 2048), (67, 2048), (9, 2056),
          (50, 128), (61, 129), (40, 256), (3, 4096), (2, 4104), (5, 8192), (3, 8200), (2, 16384), (1, 16383), (2100, 136),
          (8200, 2048), (70001, 128)]
FORMS = [(False, False, 1.0), (False, False, 0.22), (True, False, 0.5), (False, True, 1.0), (True, True, 0.5)]


@pytest.mark.parametrize("gate,post,scale", FORMS)
@pytest.mark.parametrize("T,C", SHAPES)
def test_forward(P, T, C, gate, post, scale):
    t = torch()
    for (dtype, wdtype), kind, pad in itertools.product(
            ((t.bfloat16, t.bfloat16), (t.float32, t.float32), (t.bfloat16, t.float32)), (P.LAYER_NORM, P.RMS_NORM), (0, 8, 3)):
        say(f"[residual] {T}x{C} {dtype} {wdtype} kind {kind} pad {pad} gate {gate} post {post} scale {scale}")
        h, x, vec = inputs(T, C, dtype, wdtype, kind, gate, post, T + C)
        out, y0 = strided(t.zeros_like(x), pad), strided(t.zeros_like(x), pad)
        y, h_out, mean, rstd, pm, pr = P.puro_residual_norm(strided(h, pad), strided(x, pad), **vec, kind=kind, scale=scale,
                                                           h_out=out, y=y0)
        assert y is y0 and h_out is out
        total, bound, stats = sum_reference(h, x, vec, scale, kind)
        near(h_out, total, bound + half_step(total.abs() + bound, dtype), "h_out")
        y1, m1, r1 = P.puro_layer_norm(h_out, vec["weight"], vec["bias"], kind=kind)
        assert t.equal(y, y1) and t.equal(rstd, r1) and (mean is None if kind else t.equal(mean, m1))
        if stats is None:
            assert pm is None and pr is None
        else:
            near(pr, stats[1], stats[1] * stats[3], "post_rstd")
            assert pm is None if kind else True
            if kind == 0:
                near(pm, stats[0], stats[2], "post_mean")


@pytest.mark.parametrize("T,C", [(1, 128), (17, 640), (70, 2048), (5, 4096), (3, 16384), (16390, 640), (128, 384), (4096, 2048)])
def test_codes(P, T, C):
    """The codes of both forms are the norm's own of h_out, and h_out is the tensor form's."""
    t = torch()
    for dtype, kind, (gate, post, scale) in itertools.product((t.bfloat16, t.float32), (0, 1), FORMS):
        say(f"[residual codes] {T}x{C} {dtype} kind {kind} gate {gate} post {post}")
        h, x, vec = inputs(T, C, dtype, t.bfloat16, kind, gate, post, T + C)
        y, ref, m, r, pm, pr = P.puro_residual_norm(h, x, **vec, kind=kind, scale=scale)
        rstd, prs = t.empty(T, device="cuda"), t.empty(T, device="cuda") if post else None
        q, s, h_out = P.puro_residual_norm_quant(strided(h, 16), strided(x, 16), **vec, kind=kind, scale=scale, rstd=rstd,
                                                 post_rstd=prs, h_out=strided(t.zeros_like(x), 16))
        assert t.equal(h_out, ref) and t.equal(rstd, r) and (prs is None or t.equal(prs, pr))
        q1, s1 = P.puro_layer_norm_quant(ref, vec["weight"], vec["bias"], kind=kind)
        assert t.equal(q, q1) and t.equal(s, s1)
        if T % 128:
            continue
        q, s, qT, sT, h_out, m2, r2, pm2, pr2 = P.puro_residual_norm_quant_dual(h, x, **vec, kind=kind, scale=scale)
        want = P.puro_layer_norm_quant_dual(ref, vec["weight"], vec["bias"], kind=kind)
        assert t.equal(h_out, ref) and all(t.equal(a, b) for a, b in zip((q, s, qT, sT), want))
        assert t.equal(r2, r) and (kind or t.equal(m2, m)) and (not post or t.equal(pr2, pr)) and (kind or not post or t.equal(pm2, pm))


def backward_reference(dy, dho, h_out, x, vec, stats, scale, kind):
    """The six results in 64 bits and their bounds (None where there is none)."""
    mean, rstd, pm, pr = stats
    T = x.shape[0]
    n = 47 + T / 256

    def norm_back(g, e, v, m, r):
        """The norm's backward pass of g (off by e) at v: (dx, bound, xh)."""
        m, r = (m.double()[:, None] if kind == 0 else 0.0), r.double()[:, None]
        xh = (v.double() - m) * r
        c1 = g.mean(1, keepdim=True) if kind == 0 else 0 * r
        c2 = (g * xh).mean(1, keepdim=True)
        a1, a2 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
        b = U * r * (6 * g.abs() + 54 * a1 * (1 if kind == 0 else 0) + 58 * xh.abs() * a2 + 6 * (xh * c2).abs() + 3 * abs(c1))
        b = b + r * (e + (e.mean(1, keepdim=True) if kind == 0 else 0) + xh.abs() * (e * xh.abs()).mean(1, keepdim=True))
        return r * (g - c1 - xh * c2), b, xh

    dy = dy.double()
    D, dD, xh = norm_back(dy * vec["weight"].double(), 0 * dy, h_out, mean, rstd)
    if dho is not None:
        D, dD = D + dho.double(), dD + 2 * U * dho.double().abs()
    dD = dD + U * D.abs()
    f = scale * one(vec["gate"])
    g = D * f
    if vec["post_weight"] is None:
        q = p = x.double()
        dx, bx = g, abs(f) * dD + 4 * U * g.abs()
        dpost = bpost = None
    else:
        w = vec["post_weight"].double()
        dx, bx, q = norm_back(g * w, abs(f * w) * dD + 4 * U * (g * w).abs(), x, pm, pr)
        p = q * w
        dpost, bpost = (g * q).sum(0), n * U * (g * q).abs().sum(0) + (abs(f) * dD * q.abs()).sum(0)
    dgate = bgate = None
    if vec["gate"] is not None:
        dgate = scale * (D * p).sum(0)
        bgate = abs(scale) * (n * U * (D * p).abs().sum(0) + (dD * p.abs()).sum(0))
    return ((D, dx, (dy * xh).sum(0), dy.sum(0), dgate, dpost),
            (dD, bx, n * U * (dy * xh).abs().sum(0), n * U * dy.abs().sum(0), bgate, bpost))


@pytest.mark.parametrize("gate,post,scale", FORMS)
@pytest.mark.parametrize("T,C", [(1, 1), (1, 8), (2, 7), (17, 100), (90, 128), (200, 200), (65, 512), (300, 1000), (40, 2048), (513, 2048),
                                 (33, 4100), (9, 8192), (1, 16384), (19, 16376), (4500, 256), (6001, 2048), (1300, 8192),
                                 (40000, 120), (20000, 8200), (3, 12288), (600, 12280), (70, 12281), (2, 12289), (300, 14000)])
def test_backward(P, T, C, gate, post, scale):
    t = torch()
    types = ((t.bfloat16, t.bfloat16), (t.float32, t.float32), (t.bfloat16, t.float32))
    for (dtype, wdtype), kind, pad in itertools.product(types[:2] if T * C > 1 << 24 else types, (0, 1), (0, 8, 5)):
        if T * C > 1 << 24 and pad == 8:
            continue
        say(f"[residual backward] {T}x{C} {dtype} {wdtype} kind {kind} pad {pad} gate {gate} post {post} scale {scale}")
        h, x, vec = inputs(T, C, dtype, wdtype, kind, gate, post, T + C)
        dy, dho = ((t.randn((T, C), device="cuda") * 1e-2).to(dtype) for _ in range(2))
        _, h_out, *stats = P.puro_residual_norm(h, x, **vec, kind=kind, scale=scale)
        how = dict(gate=vec["gate"], post_weight=vec["post_weight"], post_mean=stats[2], post_rstd=stats[3], scale=scale, kind=kind)
        mine = dict(x=x, dh_out=dho, **how)
        got = P.puro_residual_norm_backward(strided(dy, pad), strided(h_out, pad), vec["weight"], *stats[:2], x=strided(x, pad),
                                            dh_out=strided(dho, pad), dh=strided(t.zeros_like(x), pad),
                                            dx=strided(t.zeros_like(x), pad), **how)
        ref, bound = backward_reference(dy, dho, h_out, x, vec, stats, scale, kind)
        for what, a, b, e in zip(("dh", "dx", "dweight", "dbias", "dgate", "dpost_weight"), got, ref, bound):
            if b is None:
                assert a is None, what
                continue
            near(a, b, e + (half_step(b.abs() + e, dtype) if what in ("dh", "dx") else 1e-40), what)
        # the same call on contiguous rows, and what it may leave out
        plain = P.puro_residual_norm_backward(dy, h_out, vec["weight"], *stats[:2], **mine)
        if not pad:
            assert all(a is None and b is None or t.equal(a, b) for a, b in zip(got, plain))
        assert (plain[0] is plain[1]) == (not gate and not post and scale == 1.0)
        no_bias = P.puro_residual_norm_backward(dy, h_out, vec["weight"], *stats[:2], with_bias=False, **mine)
        assert no_bias[3] is None and all(a is None and b is None or t.equal(a, b)
                                          for k, (a, b) in enumerate(zip(no_bias, plain)) if k != 3)
        # adding to gradients that are there: one fp32 addition per element
        base = [None if v is None else t.randn(C, device="cuda") for v in plain[2:]]
        into = [None if v is None else v.clone() for v in base]
        P.puro_residual_norm_backward(dy, h_out, vec["weight"], *stats[:2], dweight=into[0], dbias=into[1], dgate=into[2],
                                      dpost_weight=into[3], accumulate=True, **mine)
        for a, b, c in zip(into, base, plain[2:]):
            assert a is None or t.equal(a, b + c)
        # in place: dh over dy, dx over x
        dyc, xc = dy.clone(), x.clone()
        P.puro_residual_norm_backward(dyc, h_out, vec["weight"], *stats[:2], **{**mine, "x": xc}, dh=dyc, dx=xc)
        assert t.equal(dyc, plain[0]) and t.equal(xc, plain[1])
        # no gradient from behind is a gradient of zero
        none = P.puro_residual_norm_backward(dy, h_out, vec["weight"], *stats[:2], **{**mine, "dh_out": None})
        zero = P.puro_residual_norm_backward(dy, h_out, vec["weight"], *stats[:2], **{**mine, "dh_out": t.zeros_like(dy)})
        assert all(a is None and b is None or t.equal(a, b) for a, b in zip(none, zero))


def test_backward_against_differences(P):
    """The derivative of sum(dy y) + sum(dh_out h_out) along random directions, by central differences of the 64-bit formula:
    the step 1e-5 leaves its square and 64-bit roundings / 1e-5, both below 1e-8 of the terms' sum.  (fp32: h_out's
    rounding, 2^-24, moves the point of the backward pass by as much, which the bound's 100 u cover as another rounding.)"""
    t = torch()
    T, C, scale = 9, 200, 0.5
    for kind, (gate, post, _) in itertools.product((0, 1), FORMS):
        h, x, vec = inputs(T, C, t.float32, t.float32, kind, gate, post, 11)
        dy, dho = t.randn_like(x), t.randn_like(x)
        _, h_out, m, r, pm, pr = P.puro_residual_norm(h, x, **vec, kind=kind, scale=scale)
        dh, dx, dw, db, dg, dp = P.puro_residual_norm_backward(
            dy, h_out, vec["weight"], m, r, x=x, gate=vec["gate"], post_weight=vec["post_weight"], post_mean=pm, post_rstd=pr,
            dh_out=dho, scale=scale, kind=kind)
        point = [h.double(), x.double(), vec["weight"].double(), t.zeros(C, dtype=t.float64, device="cuda"),
                 one(vec["gate"]) * t.ones(C, dtype=t.float64, device="cuda"),
                 one(vec["post_weight"]) * t.ones(C, dtype=t.float64, device="cuda")]

        def f(h, x, w, b, g, pw):
            def norm(v):
                d = v - v.mean(1, keepdim=True) if kind == 0 else v
                return d * (d.square().mean(1, keepdim=True) + EPS).rsqrt()
            s = h + scale * g * (norm(x) * pw if post else x)
            return dy.double() * (norm(s) * w + b), dho.double() * s
        for k, grad in enumerate((dh, dx, dw, db, dg, dp)):
            if grad is None:
                continue
            step = t.randn_like(point[k])
            ends = [f(*[v + e * step if i == k else v for i, v in enumerate(point)]) for e in (1e-5, -1e-5)]
            diff = sum(float((a - b).sum()) for a, b in zip(*ends)) / 2e-5
            got = float((grad.double() * step).sum())
            size = float((grad.double() * step).abs().sum()) + sum(float(v.abs().sum()) for v in ends[0])
            assert abs(diff - got) <= (100 * U + 1e-7) * size, (kind, gate, post, k, diff, got)


@pytest.mark.parametrize("T,C,gated", [(262144, 4104, False), (1 << 20, 2000, True), (262144, 8200, True), ((1 << 23) + 5, 8, True)])
def test_sums_of_terms_that_round_one_way(P, T, C, gated):
    """Terms of 1 + 2^-15 - 2^-23 (see tests/test_gpu_norm_sums.py, whose bound this is: it does not grow with the rows)."""
    t = torch()
    say(f"[residual sums] {T}x{C} gated {gated}")
    bound = (64 + 64 + 32 + 16 + 16 + 3) * U
    term = 1 + 2.0 ** -15 - 2.0 ** -23
    ones = t.ones((T, C), device="cuda")
    v = t.full((T, C), term, device="cuda")
    w, stat = t.ones(C, device="cuda"), t.ones(T, device="cuda")
    # dweight, dbias: dy = term at xh = 1 (mean 0).  D = rstd (u - mean(u) - xh mean(u xh)) + dh_out with u = 0 for w = 0: the gate's
    # terms are dh_out x = term
    zero = t.zeros(T, device="cuda")
    got = P.puro_residual_norm_backward(v, ones, t.zeros(C, device="cuda"), zero, stat, x=ones if gated else None,
                                        gate=w if gated else None, dh_out=v, dh=ones if not gated else None)
    for k in (2, 3, 4):
        if got[k] is not None:
            assert float((got[k].double() / (T * term) - 1).abs().max()) <= bound, k


def test_special_rows(P):
    """Infinities and NaN stay in their rows; a zero row; eps = 0; rows of no columns and no rows."""
    t = torch()
    for C, (gate, post, scale) in itertools.product((256, 2047, 4096, 12000), FORMS):
        h, x, vec = inputs(6, C, t.float32, t.float32, 0, gate, post, C)
        clean = P.puro_residual_norm(h, x, **vec, scale=scale)
        h2, x2 = h.clone(), x.clone()
        x2[1, C // 2] = float("inf")
        h2[2, 5] = float("nan")
        x2[3], h2[3] = 0, 0
        x2[4, C - 1] = float("nan")
        got = P.puro_residual_norm(h2, x2, **vec, scale=scale)
        for a, b in zip(got, clean):
            assert a is None and b is None or t.equal(a[0], b[0]) and t.equal(a[5], b[5])
        y, h_out, mean, rstd = got[:4]
        assert y[1].isnan().any() and y[2].isnan().all() and y[4].isnan().all() and mean[2].isnan()
        assert t.equal(h_out[3], t.zeros(C, device="cuda")) and t.equal(y[3], vec["bias"])
        dy = t.randn_like(h)
        args = dict(gate=vec["gate"], post_weight=vec["post_weight"], scale=scale, post_mean=got[4], post_rstd=got[5], dh_out=dy)
        dh, dx, *_ = P.puro_residual_norm_backward(dy, h_out, vec["weight"], mean, rstd, x=x2, **args)
        args.update(post_mean=clean[4], post_rstd=clean[5])
        dh1, dx1, *_ = P.puro_residual_norm_backward(dy, clean[1], vec["weight"], clean[2], clean[3], x=x, **args)
        for k in (0, 5):
            assert t.equal(dh[k], dh1[k]) and t.equal(dx[k], dx1[k])
        assert dh[2].isnan().all() and dh[3].isfinite().all() and dx[3].isfinite().all()
    for T, C in ((0, 64), (3, 0)):
        e, w = t.empty((T, C), device="cuda"), t.ones(C, device="cuda")
        y, h_out, mean, rstd, pm, pr = P.puro_residual_norm(e, e, w, gate=w, post_weight=w)
        assert y.shape == h_out.shape == (T, C) and mean.shape == (T,) and pr.isnan().all() and rstd.isnan().all()
    w, s, e = t.ones(64, device="cuda"), t.empty(0, device="cuda"), t.empty((0, 64), device="cuda")
    sums = [t.ones(64, device="cuda") for _ in range(4)]
    args = dict(x=e, gate=w, post_weight=w, post_mean=s, post_rstd=s, dweight=sums[0], dbias=sums[1], dgate=sums[2],
                dpost_weight=sums[3])
    P.puro_residual_norm_backward(e, e, w, s, s, **args, accumulate=True)
    assert all((v == 1).all() for v in sums)
    P.puro_residual_norm_backward(e, e, w, s, s, **args)
    assert all((v == 0).all() for v in sums)


def test_gaps_and_in_place(P):
    """What lies between the rows stays; h_out over h and y over x give the same bits, at every width class."""
    t = torch()
    big = [t.full((5, 131), 7.0, dtype=t.bfloat16, device="cuda") for _ in range(2)]
    h, x, vec = inputs(5, 100, t.bfloat16, t.float32, 0, True, True, 3)
    P.puro_residual_norm(h, x, **vec, h_out=big[0][:, 3:103], y=big[1][:, 3:103])
    for b in big:
        assert (b[:, :3] == 7).all() and (b[:, 103:] == 7).all() and (b[:, 3:103] != 7).any()
    for C, (gate, post, scale), dtype in itertools.product((100, 128, 1000, 2048, 8192, 16384), FORMS, (t.float32, t.bfloat16)):
        h, x, vec = inputs(3000 if C == 2048 else 37, C, dtype, dtype, 0, gate, post, 4)
        want = P.puro_residual_norm(h, x, **vec, scale=scale)
        a, b = h.clone(), x.clone()
        got = P.puro_residual_norm(a, b, **vec, scale=scale, h_out=a, y=b)
        assert got[0] is b and got[1] is a and all(p is None and q is None or t.equal(p, q) for p, q in zip(want, got))
        a, b = h.clone(), x.clone()
        got = P.puro_residual_norm(a, b, **vec, scale=scale, h_out=b, y=a)
        assert all(p is None and q is None or t.equal(p, q) for p, q in zip(want, got))
        if C % 128 == 0:
            a = h.clone()
            q, s, same = P.puro_residual_norm_quant(a, x, **vec, scale=scale, h_out=a)
            q1, s1 = P.puro_layer_norm_quant(want[1], vec["weight"], vec["bias"])
            assert same is a and t.equal(a, want[1]) and t.equal(q, q1) and t.equal(s, s1)


def calls(P, h, x, dy, vec, scale=0.5, **stream):
    t = torch()
    y, h_out, m, r, pm, pr = P.puro_residual_norm(h, x, **vec, scale=scale, **stream)
    back = P.puro_residual_norm_backward(dy, h_out, vec["weight"], m, r, x=x, gate=vec["gate"], post_weight=vec["post_weight"],
                                         post_mean=pm, post_rstd=pr, dh_out=dy, scale=scale, **stream)
    rows = P.puro_residual_norm_quant(h, x, **vec, scale=scale, **stream)
    both = P.puro_residual_norm_quant_dual(h, x, **vec, scale=scale, **stream)
    return [v for v in (y, h_out, m, r, pm, pr, *back, *rows, *both) if v is not None]


def test_streams_and_graphs(P):
    """On another stream (an object and a handle), on two at once, and captured: every replay, with other inputs and eager work
    in between, gives the eager result."""
    t = torch()
    work = []
    for k in range(2):
        h, x, vec = inputs(384, 2048, t.bfloat16, t.bfloat16, 0, True, True, 5 + k)
        dy = t.randn_like(h)
        work.append((h, x, dy, vec, calls(P, h, x, dy, vec)))
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    t.cuda.synchronize()
    got = []
    for n in range(6):
        for s, (h, x, dy, vec, want) in zip(streams, work):
            got.append((calls(P, h, x, dy, vec, stream=s if n % 2 else s.cuda_stream), want))
    t.cuda.synchronize()
    for a, b in got:
        assert all(t.equal(p, q) for p, q in zip(a, b))
    graphs = []
    for h, x, dy, vec, _ in work:                      # two graphs, each with its own workspace
        hin, xin, dyin = h.clone(), x.clone(), dy.clone()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            out = calls(P, hin, xin, dyin, vec)
        graphs.append((g, hin, xin, dyin, vec, out))
    for k in range(3):
        for (g, hin, xin, dyin, vec, out), (h, x, dy, _, _) in zip(graphs, work):
            hin.copy_(h * (k + 1))
            xin.copy_(x / (k + 1))
            dyin.copy_(dy * (2 - k))
        for g in graphs:
            g[0].replay()
        t.cuda.synchronize()
        for g, hin, xin, dyin, vec, out in graphs:
            want = calls(P, hin, xin, dyin, vec)
            assert all(t.equal(a, b) for a, b in zip(out, want)), k


def test_given_outputs_are_new_versions(P):
    t = torch()
    h, x, vec = inputs(128, 256, t.float32, t.float32, 0, True, True, 1)
    f = lambda *s: t.zeros(s, device="cuda")
    outs = {"h_out": f(128, 256), "mean": f(128), "rstd": f(128), "post_mean": f(128), "post_rstd": f(128)}
    u8 = lambda *s: t.zeros(s, dtype=t.uint8, device="cuda")
    for call, more in ((P.puro_residual_norm, {"y": f(128, 256)}), (P.puro_residual_norm_quant, {"q": u8(128, 256), "s": f(2, 128)}),
                       (P.puro_residual_norm_quant_dual, {"q": u8(128, 256), "s": f(2, 128), "qT": u8(256, 128), "sT": f(1, 256)})):
        given = {**outs, **more}
        before = {k: v._version for k, v in given.items()}
        call(h, x, **vec, **given)
        assert all(v._version > before[k] for k, v in given.items()) and h._version == x._version == 0
    grads = {"dh": f(128, 256), "dx": f(128, 256), "dweight": f(256), "dbias": f(256), "dgate": f(256), "dpost_weight": f(256)}
    before = {k: v._version for k, v in grads.items()}
    P.puro_residual_norm_backward(h, outs["h_out"], vec["weight"], outs["mean"], outs["rstd"], x=x, gate=vec["gate"],
                                  post_weight=vec["post_weight"], post_mean=outs["post_mean"], post_rstd=outs["post_rstd"], **grads)
    assert all(v._version > before[k] for k, v in grads.items())


def test_past_32_bit_offsets(P):
    """Rows more than 2^31 elements apart, read and written."""
    t = torch()
    ld = (1 << 31) + 64
    big = t.empty(2 * ld, dtype=t.bfloat16, device="cuda")
    far = lambda at: big.as_strided((2, 256), (ld, 1), at)
    h, x, vec = inputs(2, 256, t.bfloat16, t.bfloat16, 0, True, True, 9)
    y, h_out, m, r, pm, pr = P.puro_residual_norm(h, x, **vec)
    far(0).copy_(h)
    far(256).copy_(x)
    got = P.puro_residual_norm(far(0), far(256), **vec, h_out=far(512), y=far(768))
    assert all(t.equal(a, b) for a, b in zip(got, (y, h_out, m, r, pm, pr)))
    how = dict(gate=vec["gate"], post_weight=vec["post_weight"], post_mean=pm, post_rstd=pr)
    want = P.puro_residual_norm_backward(y, h_out, vec["weight"], m, r, x=x, dh_out=h, **how)
    got = P.puro_residual_norm_backward(far(768), far(512), vec["weight"], m, r, x=far(256), dh_out=far(0), dh=far(0), dx=far(768), **how)
    assert all(t.equal(a, b) for a, b in zip(got, want))


def test_past_32_bit_elements(P):
    """More than 2^31 elements: the last rows as by themselves."""
    t = torch()
    T, C = 262272, 8192
    g = t.Generator(device="cuda")
    g.manual_seed(1)
    h = t.randn((T, C), generator=g, device="cuda", dtype=t.bfloat16)
    x = t.randn((T, C), generator=g, device="cuda", dtype=t.bfloat16)
    w, gate = t.randn(C, device="cuda"), t.randn(C, device="cuda")
    tail = slice(T - 128, T)
    say(f"[residual, large] {T}x{C}")
    y, h_out, m, r, _, pr = P.puro_residual_norm(h, x, w, gate=gate, post_weight=w, kind=1)
    one = P.puro_residual_norm(h[tail], x[tail], w, gate=gate, post_weight=w, kind=1)
    assert t.equal(y[tail], one[0]) and t.equal(h_out[tail], one[1]) and t.equal(r[tail], one[3]) and t.equal(pr[tail], one[5])
    how = dict(gate=gate, post_weight=w, kind=1, with_bias=False)
    dh1, dx1, *_ = P.puro_residual_norm_backward(one[0], one[1], w, None, one[3], x=x[tail].contiguous(), post_rstd=one[5], dh_out=h[tail], **how)
    dh, dx, *sums = P.puro_residual_norm_backward(y, h_out, w, None, r, x=x, post_rstd=pr, dh_out=h, dh=y, dx=x, **how)
    assert t.equal(dh[tail], dh1) and t.equal(dx[tail], dx1) and all(s is None or s.isfinite().all() for s in sums)


def test_more_short_rows_than_a_launch_has_threads(P):
    """2^30 rows and some of one column: the rows at the end as by themselves."""
    t = torch()
    T = (1 << 30) + 77
    h = t.ones((T, 1), device="cuda", dtype=t.bfloat16)
    h[::3] = -2
    w = t.ones(1, device="cuda", dtype=t.bfloat16)
    say(f"[residual, long] {T}x1")
    tail = h[-1000:].clone()
    y1, o1, _, r1, _, _ = P.puro_residual_norm(tail, tail, w, kind=P.RMS_NORM, gate=w)
    y, o, _, r, _, _ = P.puro_residual_norm(h, h, w, kind=P.RMS_NORM, gate=w)
    assert t.equal(y[-1000:], y1) and t.equal(o[-1000:], o1) and t.equal(r[-1000:], r1) and t.equal(o, 2 * h)


def test_binding_refusals(P):
    t = torch()
    h, x, vec = inputs(4, 128, t.bfloat16, t.bfloat16, 0, True, True, 1)
    w, f = vec["weight"], t.empty(4, device="cuda")
    y = t.empty_like(h)

    def refused(error, *a, **k):
        with pytest.raises(error):
            P.puro_residual_norm(*a, **k)
    refused(TypeError, h, x.float(), w)
    refused(TypeError, h, x, w, gate=w.float())
    refused(ValueError, h, x[:3], w)
    refused(ValueError, h, x, w, gate=w[:64])
    refused(ValueError, h, x, w, post_weight=w[:64])
    refused(ValueError, h, x, w, kind=7)
    refused(ValueError, h, x, w, kind=P.RMS_NORM, mean=f)
    refused(ValueError, h, x, w, post_rstd=f)
    refused(ValueError, h, x, w, post_mean=f)
    refused(ValueError, h, x, w, kind=P.RMS_NORM, post_weight=w, post_mean=f)
    refused(ValueError, h.cpu(), x, w)
    refused(P.PuroError, h, x, w, h_out=y, y=y)
    refused(P.PuroError, h, x, w, scale=float("inf"))
    refused(P.PuroError, h, x, w, scale=float("nan"))
    refused(P.PuroError, h, x, w, eps=-1.0)
    with pytest.raises(P.PuroError):
        P.puro_residual_norm_quant_dual(h, x, w)                  # 4 rows
    with pytest.raises(P.PuroError):
        P.puro_residual_norm_quant(h[:, :100], x[:, :100], w[:100])
    back = lambda **k: P.puro_residual_norm_backward(h, h, w, f, f, **k)
    with pytest.raises(ValueError):
        back(gate=w)                                              # needs x
    with pytest.raises(ValueError):
        back(dgate=t.empty(128, device="cuda"))
    with pytest.raises(ValueError):
        back(dpost_weight=t.empty(128, device="cuda"))
    with pytest.raises(ValueError):
        back(post_rstd=f)
    with pytest.raises(ValueError):
        back(accumulate=True)
    with pytest.raises(ValueError):
        back(kind=P.RMS_NORM)
    with pytest.raises(P.PuroError):
        back(dh=y, dx=y)
    with pytest.raises(P.PuroError):
        back(scale=float("inf"))
