"""GPU tests of the rotary positions against the formula in 64 bits.

Tolerance, with u = 2^-24: the angle in quarter turns has two roundings of 64 bits, 2^-51 of the angle; what is left of it is
rounded to 32 bits (a fraction of u) and its cosine and sine are within 4 ulp, 4 u of 1; the scale has two roundings (from 64
bits, and its product).  A turned value has two products and a sum, |a c| + |b s| times 2 u.  In all
(9 u + 2^-50 |angle|) |scale| (|a| + |b|), then half a step of its type."""
import itertools

import pytest

from gpu_util import say, torch
from test_gpu_norm import half_step, near

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def frequencies(pairs, base=10000.0):
    t = torch()
    return base ** (-t.arange(pairs, dtype=t.float64, device="cuda") / max(1, pairs))


def reference(x, freqs, positions, interleaved, scale, inverse):
    t = torch()
    v, n = x.double(), freqs.numel()
    angle = positions.double()[:, None] * freqs
    c, s = t.cos(angle)[:, None] * scale, t.sin(angle)[:, None] * (-scale if inverse else scale)
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = v[..., first], v[..., second]
    y, e = v.clone(), t.zeros_like(v)
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    bound = (9 * U + 2.0 ** -50 * angle.abs())[:, None] * abs(scale) * (a.abs() + b.abs())
    e[..., first] = e[..., second] = bound
    return y, e


def tensor(T, H, D, dtype, seed, pad=0, order="thd"):
    """[T, H, D] with heads `pad` elements apart in either order, behind a gap of `pad`, in a buffer of NaN."""
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    v = t.randn((T, H, D), generator=g, device="cuda").to(dtype)
    if not pad and order == "thd":
        return v
    outer, inner = (T, H) if order == "thd" else (H, T)
    big = t.full((pad + outer * inner * (D + pad) + 8,), float("nan"), device="cuda", dtype=dtype)
    w = big[pad:][: outer * inner * (D + pad)].view(outer, inner, D + pad)[..., :D]
    w = w if order == "thd" else w.transpose(0, 1)
    w.copy_(v)
    return w


CASES = [(1, 1, 2, 1), (1, 24, 128, 64), (7, 3, 6, 3), (5, 2, 80, 16), (33, 5, 64, 20), (130, 8, 128, 64), (3, 40, 96, 33), (2, 1, 256, 128),
         (4, 2, 5, 2), (9, 3, 130, 65), (1, 3, 4096, 2048), (5, 300, 16, 8), (1000, 3, 24, 1), (2, 5, 72, 0), (4097, 1, 32, 16),
         (300, 24, 128, 64), (2, 70, 1000, 500)]


@pytest.mark.parametrize("T,H,D,pairs", CASES)
def test_turns(P, T, H, D, pairs):
    t = torch()
    for dtype, interleaved, inverse, (pad, order) in itertools.product((t.bfloat16, t.float32), (False, True), (False, True),
                                                                       ((0, "thd"), (8, "thd"), (3, "thd"), (8, "htd"))):
        say(f"[rotary] {T}x{H}x{D} pairs {pairs} {dtype} interleaved {interleaved} inverse {inverse} pad {pad} {order}")
        x = tensor(T, H, D, dtype, T + D, pad, order)
        freqs, scale = frequencies(pairs), 1.0 if pad else 1.1
        positions = t.randint(0, 40000, (T,), device="cuda")
        layout = P.ROTARY_INTERLEAVED if interleaved else P.ROTARY_HALF
        how = dict(layout=layout, scale=scale, inverse=inverse)
        out = tensor(T, H, D, dtype, 0, 8 if pad == 3 else pad, order)
        base = out._base if out._base is not None else out
        gaps = base.isnan()
        y = P.puro_rotary(x, freqs, positions, y=out, **how)
        ref, bound = reference(x, freqs, positions, interleaved, scale, inverse)
        near(y, ref, bound + (half_step(ref.abs() + bound, dtype) if pairs else 0) * (bound > 0), "turned")
        assert t.equal(y[..., 2 * pairs:], x[..., 2 * pairs:])
        assert t.equal(gaps, base.isnan()), "gaps"
        y2 = P.puro_rotary(x, freqs, positions, **how)
        assert y2.is_contiguous() and t.equal(y2, y)
        mine = x.clone(memory_format=t.preserve_format) if order == "htd" else tensor(T, H, D, dtype, T + D, pad, order)
        assert P.puro_rotary(mine, freqs, positions, y=mine, **how) is mine and t.equal(mine, y)
        # positions counted from a start
        a = P.puro_rotary(x, freqs, t.arange(T, device="cuda") + 77, **how)
        assert t.equal(a, P.puro_rotary(x, freqs, start=77, **how))


@pytest.mark.parametrize("start", [0, -5, 123456, 10 ** 7, 2 ** 31 - 4, 2 ** 40, -2 ** 45])
def test_far_positions(P, start):
    """64 bits hold the angle; in 32 it would be lost."""
    t = torch()
    for dtype, interleaved in itertools.product((t.float32, t.bfloat16), (False, True)):
        x, freqs = tensor(9, 2, 64, dtype, 3), frequencies(32, 500000.0)
        positions = t.arange(9, device="cuda") + start
        y = P.puro_rotary(x, freqs, start=start, layout=int(interleaved))
        assert t.equal(y, P.puro_rotary(x, freqs, positions, layout=int(interleaved)))
        ref, bound = reference(x, freqs, positions, interleaved, 1.0, False)
        near(y, ref, bound + half_step(ref.abs() + bound, dtype), "far")


def test_exact_quarters(P):
    """Angles at whole quarter turns of 64 bits' pi: the cosine's and the sine's zero is left to 64 bits' rounding of the angle."""
    t = torch()
    x = t.randn((9, 1, 2), device="cuda")
    freqs = t.full((1,), 3.14159265358979323846 / 2, dtype=t.float64, device="cuda")
    y = P.puro_rotary(x, freqs)
    ref, bound = reference(x, freqs, t.arange(9, device="cuda"), False, 1.0, False)
    near(y, ref, bound, "quarters")
    a, b = x[:, 0, 0], x[:, 0, 1]
    for k in range(9):
        want = [(a[k], b[k]), (-b[k], a[k]), (-a[k], -b[k]), (b[k], -a[k])][k % 4]
        assert abs(float(y[k, 0, 0] - want[0])) < 1e-6 and abs(float(y[k, 0, 1] - want[1])) < 1e-6


def test_inverse_is_the_gradient(P):
    """<turn(x), dy> = <x, inverse(dy)> within both results' bounds, and against central differences of the formula."""
    t = torch()
    for interleaved, pairs in itertools.product((False, True), (8, 20)):
        x, dy, freqs = tensor(50, 3, 40, t.float32, 1), tensor(50, 3, 40, t.float32, 2), frequencies(pairs)
        pos = t.arange(50, device="cuda") * 31
        y = P.puro_rotary(x, freqs, pos, layout=int(interleaved), scale=0.9)
        dx = P.puro_rotary(dy, freqs, pos, layout=int(interleaved), scale=0.9, inverse=True)
        by, bx = reference(x, freqs, pos, interleaved, 0.9, False)[1], reference(dy, freqs, pos, interleaved, 0.9, True)[1]
        off = abs(float((y.double() * dy.double()).sum() - (x.double() * dx.double()).sum()))
        assert off <= float((by * dy.double().abs()).sum() + (bx * x.double().abs()).sum()) + 1e-9
        step = t.randn_like(x).double()
        ends = [reference(x.double() + e * step, freqs, pos, interleaved, 0.9, False)[0] for e in (0.5, -0.5)]
        diff = float(((ends[0] - ends[1]) * dy.double()).sum())              # the turn is linear: no error of the difference
        assert abs(diff - float((dx.double() * step).sum())) <= float((bx * step.abs()).sum()) + 1e-9


def test_special_values(P):
    """NaN and infinities stay in their pair; copied columns keep their bits; repeated input (stride 0)."""
    t = torch()
    for pairs, interleaved, here in itertools.product((1, 2, 5, 13), (False, True), (False, True)):
        bits = t.randint(-2 ** 15, 2 ** 15, (3, 2, 30), device="cuda").to(t.int16)         # every NaN among them
        x = bits.view(t.bfloat16).clone()
        y = P.puro_rotary(x, frequencies(pairs), layout=int(interleaved), y=x if here else None)
        assert t.equal(y.view(t.int16)[..., 2 * pairs:], bits[..., 2 * pairs:]), (pairs, interleaved, here)
    for dtype, interleaved in itertools.product((t.float32, t.bfloat16), (False, True)):
        x = tensor(6, 2, 29, dtype, 5)
        freqs = frequencies(9)
        clean = P.puro_rotary(x, freqs, layout=int(interleaved))
        x[2, 1, 4] = float("nan")
        x[3, 0, 0] = float("inf")
        x[4, 1, 20] = float("inf")
        x[5, 0, 28] = float("nan")
        y = P.puro_rotary(x, freqs, layout=int(interleaved))
        bad = ~(y == clean)
        pair = {(2, 1, 4), (2, 1, 5 if interleaved else 13), (3, 0, 0), (3, 0, 1 if interleaved else 9), (4, 1, 20), (5, 0, 28)}
        assert {tuple(v) for v in bad.nonzero().tolist()} == pair
        assert y[4, 1, 20].isinf() and y[5, 0, 28].isnan()
        row = x[:1, :1].expand(6, 2, 29)
        assert t.equal(P.puro_rotary(row, freqs, layout=int(interleaved)), P.puro_rotary(row.contiguous(), freqs, layout=int(interleaved)))


def test_empty(P):
    t = torch()
    f = frequencies(4)
    for shape in ((0, 3, 8), (3, 0, 8)):
        assert P.puro_rotary(t.empty(shape, device="cuda"), f).shape == shape
    e = t.empty((2, 3, 0), device="cuda")
    assert P.puro_rotary(e, f[:0]).shape == e.shape


def test_streams_and_graphs(P):
    t = torch()
    x, freqs = tensor(500, 24, 128, t.bfloat16, 4), frequencies(64)
    pos = t.randint(0, 5000, (500,), device="cuda")
    want = P.puro_rotary(x, freqs, pos)
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    t.cuda.synchronize()
    got = [P.puro_rotary(x, freqs, pos, stream=streams[k % 2] if k % 3 else streams[k % 2].cuda_stream) for k in range(12)]
    t.cuda.synchronize()
    assert all(t.equal(g, want) for g in got)
    xin, pin = x.clone(), pos.clone()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        y = P.puro_rotary(xin, freqs, pin)
        z = P.puro_rotary(y, freqs, pin, inverse=True)
    for k in range(3):
        xin.copy_(x * (k + 1))
        pin.add_(k)
        graph.replay()
        t.cuda.synchronize()
        e = P.puro_rotary(xin, freqs, pin)
        assert t.equal(y, e) and t.equal(z, P.puro_rotary(e, freqs, pin, inverse=True)), k


def test_versions(P):
    t = torch()
    x, y = tensor(4, 2, 8, t.float32, 1), t.zeros((4, 2, 8), device="cuda")
    P.puro_rotary(x, frequencies(4), y=y)
    assert y._version > 0 and x._version == 0


def test_past_32_bits(P):
    """Tokens more than 2^31 elements apart, and more than 2^31 elements: the last ones as by themselves."""
    t = torch()
    ld, f = (1 << 31) + 64, frequencies(32)
    big = t.empty(2 * ld, dtype=t.bfloat16, device="cuda")
    far = lambda at: big.as_strided((2, 3, 64), (ld, 64, 1), at)
    v = tensor(2, 3, 64, t.bfloat16, 7)
    far(0).copy_(v)
    assert t.equal(P.puro_rotary(far(0), f, y=far(512)), P.puro_rotary(v, f))
    del big
    T, H, D = 1 << 20, 33, 64
    say("[rotary, large]")
    x = t.randn((T, H, D), device="cuda", dtype=t.bfloat16)
    tail = x[-100:].clone()
    y = P.puro_rotary(x, f, y=x)
    assert t.equal(y[-100:], P.puro_rotary(tail, f, start=T - 100))
    big = t.randint(-99, 99, (1, (1 << 31) - 1, 1), device="cuda", dtype=t.int8).to(t.bfloat16)     # as many heads as there may be
    assert t.equal(P.puro_rotary(big, f[:0]), big)
    del big
    x = t.randn((1 << 25, 1, 2), device="cuda", dtype=t.bfloat16)            # more tiles than workgroups of a launch
    y = P.puro_rotary(x, f[:1])
    assert t.equal(y[-100:], P.puro_rotary(x[-100:], f[:1], start=(1 << 25) - 100))
    assert t.equal(y[1 << 24:][:100], P.puro_rotary(x[1 << 24:][:100], f[:1], start=1 << 24))


def test_refusals(P):
    t = torch()
    x, f = tensor(4, 2, 16, t.float32, 1), frequencies(4)

    def refused(error, *a, **k):
        with pytest.raises(error):
            P.puro_rotary(*a, **k)
    refused(ValueError, x[0], f)
    refused(TypeError, x.half(), f)
    refused(TypeError, x, f.float())
    refused(ValueError, x, frequencies(9))
    refused(ValueError, x, f.cpu())
    refused(ValueError, x.cpu(), f)
    refused(ValueError, x, f, t.arange(3, device="cuda"))
    refused(TypeError, x, f, t.arange(4, device="cuda", dtype=t.int32))
    refused(ValueError, x, f, layout=2)
    refused(ValueError, x.transpose(1, 2), f)
    refused(TypeError, x, f, y=x.bfloat16())
    refused(ValueError, x, f, y=x[:3])
    refused(P.PuroError, x, f, scale=float("nan"))
    refused(P.PuroError, x, f, y=x[:1].expand(4, 2, 16))                     # tokens over each other
    refused(P.PuroError, x, f, y=t.empty(200, device="cuda").as_strided((4, 2, 16), (16, 16, 1)))
    same = t.empty(400, device="cuda")
    refused(P.PuroError, same.as_strided((4, 2, 16), (32, 16, 1)), f, y=same.as_strided((4, 2, 16), (16, 64, 1)))
    refused(P.PuroError, t.empty((1, 1, 2 * 2049), device="cuda"), frequencies(2049))
