"""GPU tests of the global gradient norm and clipping, against 64-bit sums.

Tolerances, with u = 2^-24: squares are exact in 64 bits and their sum is off by under 1e-10, so the norm has its
square root's and the conversion's rounding: 2 u.  The coefficient adds one of norm + 1e-6 and one of the division:
4 u; the product one more, and bf16 gradients half a step of their own."""
import math

import pytest

from gpu_util import say, torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def make(sizes, dtypes, seed, scale=1e-2, shift=0):
    """Tensors cut one behind the other out of one buffer per type, from element `shift`: every alignment occurs."""
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for n, dt in zip(sizes, dtypes):
        flat = (t.randn(n + 16, generator=g, device="cuda") * scale).to(dt)
        out.append(flat[shift % 9:][:n])
        shift += 1
    return out


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


SETS = [[1], [0], [3, 0, 5], [8192], [8193, 8191, 1], [100003], [1 << 20, 17, 4096], [5] * 300, [2048 * 2048, 2047, 2048]]


@pytest.mark.parametrize("sizes", SETS, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("types", ["fp32", "bf16", "mixed"])
def test_norm_and_clip(P, sizes, types):
    t = torch()
    dts = {"fp32": [t.float32], "bf16": [t.bfloat16], "mixed": [t.float32, t.bfloat16]}[types]
    dts = [dts[i % len(dts)] for i in range(len(sizes))]
    for shift in (0, 1, 3):
        say(f"[clip] {sizes[:4]} {types} shift {shift}")
        grads = make(sizes, dts, len(sizes) + shift, shift=shift)
        ref = norm64(grads)
        n = P.puro_grad_norm(grads)
        assert n.shape == () and abs(float(n) - ref) <= 2 * U * ref
        for max_norm in (ref * 0.37 + 1e-3, ref * 2 + 1.0, 0.0):
            outs = [t.full((g.numel() + 5,), 9.0, device="cuda", dtype=g.dtype)[(i + shift) % 4:][: g.numel()]
                    for i, g in enumerate(grads)]
            norm, got = P.puro_clip_grad_norm(grads, max_norm, outs=outs)
            assert float(norm) == float(n) and got is outs
            coef = min(1.0, max_norm / (ref + 1e-6))
            for g, o in zip(grads, outs):
                want = g.double() * coef
                step = t.finfo(g.dtype).eps / 2 if g.dtype == t.bfloat16 else 0.0
                assert ((o.double() - want).abs() <= want.abs() * (6 * U + step * (1 + 2.0 ** -7)) + 1e-40).all()
                base = o._base
                if base is not None and o.numel():
                    lo = o.storage_offset()
                    assert (base[:lo] == 9).all() and (base[lo + o.numel():] == 9).all()
            # in place gives the same bits, and a norm handed in does too
            mine, other = [g.clone() for g in grads], [g.clone() for g in grads]
            _, same = P.puro_clip_grad_norm(mine, max_norm)
            P.puro_scale_by_norm(other, max_norm, norm)
            for a, b, c in zip(mine, other, outs):
                assert t.equal(a, c) and t.equal(b, c)


def test_range_and_non_finite(P):
    """Squares beyond fp32's range at both ends; a norm that is not finite is passed on."""
    t = torch()
    big = t.full((1000,), 1e30, device="cuda")
    small = t.full((1000,), 1e-30, device="cuda")
    assert abs(float(P.puro_grad_norm([big])) / (float(big[0]) * math.sqrt(1000)) - 1) <= 4 * U
    assert abs(float(P.puro_grad_norm([small])) / (float(small[0]) * math.sqrt(1000)) - 1) <= 4 * U
    n, _ = P.puro_clip_grad_norm([big], 1.0)
    assert abs(float(P.puro_grad_norm([big])) - 1) < 1e-5
    g = t.ones(5000, device="cuda")
    g[77] = float("inf")
    n, (o,) = P.puro_clip_grad_norm([g], 1.0)
    assert n.isinf() and o[77].isnan() and (o[:77] == 0).all() and (o[78:] == 0).all()
    g = t.ones(5000, device="cuda")
    g[78] = float("nan")
    n, (o,) = P.puro_clip_grad_norm([g, ], 1.0)
    assert n.isnan() and o.isnan().all()
    z = t.zeros(100, device="cuda")
    n, (o,) = P.puro_clip_grad_norm([z], 1.0)
    assert float(n) == 0 and (o == 0).all()
    n, (o,) = P.puro_clip_grad_norm([t.ones(100, device="cuda")], math.inf)
    assert float(n) == 10 and (o == 1).all()


def test_more_than_32_bits_of_elements(P):
    t = torch()
    n = 2 ** 31 + 5
    g = t.ones(n, dtype=t.bfloat16, device="cuda")
    norm, _ = P.puro_clip_grad_norm([g[:7].clone(), g], 1024.0)
    ref = math.sqrt(n + 7)
    assert abs(float(norm) - ref) <= 2 * U * ref
    want = float(t.tensor(1024.0 / (ref + 1e-6)).bfloat16())
    for part in (g[:1000], g[2 ** 30: 2 ** 30 + 1000], g[-1000:]):
        assert (part == want).all()
    assert int((g != want).sum()) == 0


def test_no_tensors_and_empty_ones(P):
    t = torch()
    assert float(P.puro_grad_norm([])) == 0
    n, o = P.puro_clip_grad_norm([], 1.0)
    assert float(n) == 0 and o == []
    n, o = P.puro_clip_grad_norm([t.empty(0, device="cuda")], 1.0)
    assert float(n) == 0


def test_refusals(P):
    t = torch()
    g = t.ones(64, 64, device="cuda")
    with pytest.raises(ValueError):
        P.puro_grad_norm([g[:, :32]])
    with pytest.raises(ValueError):
        P.puro_grad_norm([g[:1].expand(64, 64)])
    with pytest.raises(ValueError):
        P.puro_clip_grad_norm([g.t()], 1.0, outs=[t.empty_like(g).contiguous()])
    with pytest.raises(ValueError):
        P.puro_clip_grad_norm([g], 1.0, outs=[t.ones(64, device="cuda")])
    with pytest.raises(TypeError):
        P.puro_clip_grad_norm([g], 1.0, outs=[g.bfloat16()])
    with pytest.raises(TypeError):
        P.puro_clip_grad_norm([g], 1.0, outs=[None])
    with pytest.raises(ValueError):
        P.puro_clip_grad_norm([g.cpu()], 1.0)
    with pytest.raises(P.PuroError):
        P.puro_clip_grad_norm([g, g], 1.0)
    with pytest.raises(P.PuroError):
        P.puro_clip_grad_norm([g], -1.0)
    with pytest.raises(P.PuroError):
        P.puro_clip_grad_norm([g], 1.0, workspace=t.empty(4, dtype=t.uint8, device="cuda"))
    with pytest.raises(ValueError):
        P.puro_scale_by_norm([g], 1.0, t.ones(2, device="cuda"))
    assert (g == 1).all()


def test_other_orders_of_dimensions(P):
    """A dense tensor in another order of its dimensions: the same norm and the same elements."""
    t = torch()
    g = t.randn((3, 50, 70), device="cuda").permute(2, 0, 1)
    n, (o,) = P.puro_clip_grad_norm([g], 0.5, outs=[t.empty_like(g)])
    n2, (o2,) = P.puro_clip_grad_norm([g.contiguous()], 0.5)
    assert float(n) == float(n2) and t.equal(o, o2)
    P.puro_clip_grad_norm([g], 0.5)
    assert t.equal(g, o)


def test_graph_and_stream(P):
    t = torch()
    grads = make([5000, 70000, 3], [t.float32, t.bfloat16, t.float32], 5)
    keep = [g.clone() for g in grads]
    outs = [t.empty_like(g) for g in grads]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    n1, _ = P.puro_clip_grad_norm(grads, 0.5, outs=outs, stream=side)
    t.cuda.synchronize()
    n0, want = P.puro_clip_grad_norm(grads, 0.5, outs=[t.empty_like(g) for g in grads])
    assert float(n0) == float(n1) and all(t.equal(a, b) for a, b in zip(outs, want))
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        gn, _ = P.puro_clip_grad_norm(grads, 0.5)
    for k in range(3):
        for g, s in zip(grads, keep):
            g.copy_(s * (k + 1))
        eager = [g.clone() for g in grads]
        en, _ = P.puro_clip_grad_norm(eager, 0.5)
        graph.replay()
        t.cuda.synchronize()
        assert float(gn) == float(en) and all(t.equal(a, b) for a, b in zip(grads, eager)), k


def test_clip_grad_norm_takes_main_grads_and_each_parameter_once(P):
    t = torch()
    from blockwise_scaled_fp8_quant_amd.clip import clip_grad_norm_, gradients
    a = t.nn.Parameter(t.ones(300, device="cuda", dtype=t.bfloat16))
    b = t.nn.Parameter(t.ones(300, device="cuda"))
    c = t.nn.Parameter(t.ones(5, device="cuda"))
    a.main_grad = t.full((300,), 2.0, device="cuda")
    b.grad = t.full((300,), 1.0, device="cuda")
    assert [g.data_ptr() for g in gradients([a, b, c, a])] == [a.main_grad.data_ptr(), b.grad.data_ptr()]
    n = clip_grad_norm_([a, b, c, a], 1.0)
    ref = math.sqrt(300 * 5)
    assert abs(float(n) - ref) <= 2 * U * ref
    assert (a.main_grad - 2 / (ref + 1e-6)).abs().max() <= 2 / ref * 6 * U
    assert float(clip_grad_norm_([c], 1.0)) == 0
    assert abs(float(clip_grad_norm_(b, 1e9)) - math.sqrt(300) / ref) <= 1e-5
