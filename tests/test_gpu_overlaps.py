"""GPU tests of tensors that lie within each other's spans: columns side by side in one buffer and outputs in their inputs' places
give the results of separate tensors, bit for bit; what shares memory otherwise is refused and nothing is written."""
import itertools
import random

import pytest

from gpu_util import say, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def same(a, b):
    return all((x is None) == (y is None) and (x is None or torch().equal(x, y)) for x, y in zip(a, b))


def vectors(C, dtype):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(C)
    return [(1 + 0.1 * t.randn(C, generator=g, device="cuda")).to(dtype) for _ in range(3)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,C", [(300, 256), (5, 37), (1, 8)])
def test_columns_of_one_buffer(P, T, C, dtype):
    """h, x, h_out and y, then dy, dh and dx, as neighbouring columns of one wide buffer."""
    t = torch()
    dt = getattr(t, dtype)
    w, gate, post = vectors(C, dt)
    say(f"[overlaps] {T} x {C} {dtype}")
    wide = t.randn((T, 7 * C), device="cuda").to(dt)
    part = [wide[:, i * C: (i + 1) * C] for i in range(7)]
    h, x, dy = (part[i].clone() for i in (0, 1, 4))
    how = dict(kind=1, gate=gate, post_weight=post, scale=0.5)
    want = P.puro_residual_norm(h, x, w, **how)
    got = P.puro_residual_norm(part[0], part[1], w, h_out=part[2], y=part[3], **how)
    assert same(got, want) and t.equal(part[0], h) and t.equal(part[1], x)
    back = lambda dy, h_out, x, **k: P.puro_residual_norm_backward(dy, h_out, w, None, want[3], x=x, post_rstd=want[5], dh_out=dy,
                                                                   with_bias=False, **how, **k)
    want_back = back(dy, want[1], x)
    got = back(part[4], part[2], part[1], dh=part[5], dx=part[6])
    assert same(got, want_back) and t.equal(part[4], dy) and t.equal(part[2], want[1]) and t.equal(part[1], x)


@pytest.mark.parametrize("T,C,dtype", [(300, 256, "bfloat16"), (70, 2047, "bfloat16"), (65, 5000, "float32"), (70, 9000, "bfloat16"),
                                       (70, 12800, "bfloat16")])
@pytest.mark.parametrize("gated", [True, False])
def test_gradients_in_their_inputs_places(P, T, C, dtype, gated):
    """dh and dx each in the place of dy, h_out, dh_out or x (not both of one)."""
    t = torch()
    dt = getattr(t, dtype)
    w, gate, post = vectors(C, dt)
    how = dict(gate=gate, post_weight=post) if gated else {}
    given = {k: (t.randn((T, C), device="cuda") + 0.2).to(dt) for k in ("dy", "h_out", "dh_out", "x")}
    f = lambda v: v.float().square().mean(1).add(1e-5).rsqrt()
    rstd, prstd = f(given["h_out"]), f(given["x"])

    def run(v, **k):
        return P.puro_residual_norm_backward(v["dy"], v["h_out"], w, None, rstd, x=v["x"], post_rstd=prstd if gated else None,
                                             dh_out=v["dh_out"], scale=0.5, kind=1, with_bias=False, **how, **k)
    want = run(given)
    for a, b in itertools.permutations((*given, None), 2):
        mine = {k: v.clone() for k, v in given.items()}
        got = run(mine, dh=mine.get(a), dx=mine.get(b))
        assert same(got, want), (a, b)
        for k in given:
            assert k in (a, b) or t.equal(mine[k], given[k])


def test_rows_that_interleave(P):
    """h_out laid over h at random, strides its own: refused with nothing written where a cell is in both, else the result."""
    t = torch()
    rng = random.Random(5)
    n, clear, clash = 400, 0, 0
    for _ in range(400):
        T, C = rng.randint(1, 6), rng.randint(1, 8)
        ld, other = C + rng.randint(0, 12), 0
        other = ld if rng.random() < 0.5 else C + rng.randint(0, 20)
        a, b = rng.randint(0, 60), rng.randint(0, 120)
        buffer = t.randn(n, device="cuda")
        before = buffer.clone()
        h, out = buffer.as_strided((T, C), (ld, 1), a), buffer.as_strided((T, C), (other, 1), b)
        x, w = t.randn((T, C), device="cuda"), t.ones(C, device="cuda")
        cells = lambda at, ld: {at + i * ld + c for i in range(T) for c in range(C)}
        inside = a == b and (T == 1 or ld == other)
        if cells(a, ld) & cells(b, other) and not inside:
            clash += 1
            with pytest.raises(P.PuroError):
                P.puro_residual_norm(h, x, w, kind=1, h_out=out)
            assert t.equal(buffer, before)
        else:
            clear += 1
            want = P.puro_residual_norm(h.clone(), x, w, kind=1)
            assert same(P.puro_residual_norm(h, x, w, kind=1, h_out=out), want)
    assert clear > 50 and clash > 50


def test_refusals_write_nothing(P):
    t = torch()
    h, x, w = t.randn((64, 256), device="cuda"), t.randn((64, 256), device="cuda"), t.ones(256, device="cuda")
    kept = [v.clone() for v in (h, x, w)]
    rstd = t.ones(64, device="cuda")
    two = t.zeros(300, device="cuda")
    calls = [lambda: P.puro_residual_norm(h, x, w, kind=1, y=h, h_out=h), lambda: P.puro_residual_norm(h, x, w, kind=1, rstd=h.view(-1)[5:69]),
             lambda: P.puro_residual_norm_quant(h, x, w, kind=1, q=h.view(t.uint8)[:, :256]),
             lambda: P.puro_residual_norm_quant(h, x, w, kind=1, h_out=h, s=h.view(-1)[:128].view(2, 64)),
             lambda: P.puro_residual_norm_backward(h, x, w, None, rstd, kind=1, dweight=two[:256], dbias=two[44:]),
             lambda: P.puro_residual_norm_backward(h, x, w, None, rstd, kind=1, dweight=w),
             lambda: P.puro_residual_norm_backward(h, x, w, None, rstd, kind=1, workspace=x)]
    for k, call in enumerate(calls):
        with pytest.raises(P.PuroError):
            call()
            raise AssertionError(f"call {k} was not refused")
    assert all(t.equal(a, b) for a, b in zip((h, x, w), kept)) and not two.any()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_heads_of_one_buffer(P, dtype):
    """A turned half of the heads beside the given one, tokens or heads outermost, or a part of every head beside the rest."""
    t = torch()
    dt = getattr(t, dtype)
    freqs = t.logspace(0, -3, 8, dtype=t.float64, device="cuda")
    for shape, cut in (((50, 8, 32), lambda b, k: b[:, 4 * k: 4 * k + 4]), ((50, 8, 32), lambda b, k: b[:, k::2]),
                       ((8, 50, 32), lambda b, k: b.transpose(0, 1)[:, 4 * k: 4 * k + 4]), ((50, 4, 64), lambda b, k: b[..., 32 * k: 32 * k + 32]),
                       ((1, 8, 32), lambda b, k: b[:, 4 * k: 4 * k + 4]), ((50, 1, 64), lambda b, k: b[..., 32 * k: 32 * k + 32])):
        say(f"[overlaps] heads {shape} {dtype}")
        b = t.randn(shape, device="cuda").to(dt)
        x = cut(b, 0).clone()
        for layout in (0, 1):
            want = P.puro_rotary(x, freqs, layout=layout)
            assert t.equal(P.puro_rotary(cut(b, 0), freqs, layout=layout, y=cut(b, 1)), want) and t.equal(cut(b, 0), x)


def test_heads_that_interleave(P):
    """x and y laid over each other at random: refused with nothing written where a cell is in both, else the result."""
    t = torch()
    rng = random.Random(6)
    freqs = t.ones(1, dtype=t.float64, device="cuda")
    clear = clash = 0
    for _ in range(400):
        T, H, D = rng.randint(1, 4), rng.randint(1, 4), rng.randint(2, 6)
        inner = D + rng.randint(0, 8)
        outer = (max(T, H) - 1) * inner + D + rng.randint(0, 20)
        ldy = (outer, inner) if rng.random() < 0.5 else (inner, outer)
        ldx = ldy if rng.random() < 0.6 else (rng.randint(0, 30), rng.randint(0, 30))
        a, b = rng.randint(0, 120), rng.randint(0, 120)
        buffer = t.randn(600, device="cuda")
        before = buffer.clone()
        x, y = buffer.as_strided((T, H, D), (*ldx, 1), a), buffer.as_strided((T, H, D), (*ldy, 1), b)
        cells = lambda at, ld: {at + i * ld[0] + k * ld[1] + d for i in range(T) for k in range(H) for d in range(D)}
        inside = a == b and (T == 1 or ldx[0] == ldy[0]) and (H == 1 or ldx[1] == ldy[1])
        if cells(a, ldx) & cells(b, ldy) and not inside:
            clash += 1
            with pytest.raises(P.PuroError):
                P.puro_rotary(x, freqs, y=y)
            assert t.equal(buffer, before)
        else:
            clear += 1
            want = P.puro_rotary(x.clone(memory_format=t.contiguous_format), freqs)
            assert t.equal(P.puro_rotary(x, freqs, y=y), want)
    assert clear > 50 and clash > 50
