"""GPU tests of the AdamW step over many tensors, with fp32 and 8-bit states.

8-bit states are held to the oracle (oracle/adamw.py), which rounds operation by operation: codes and scales are equal to the
bit.  Everything else is held to the formula in 64 bits.  Tolerances, with u = 2^-24; with clipping the factor has 4 u
(norm + 1e-6, the quotient, max_norm and the norm itself), g one more:
    m'   each product has two roundings (the factor's from 64 bits, its own), the sum one: 2 u |b1 m| + 7 u |c1 g| + u |m'|
    v'   2 u |b2 v| + 13 u c2 g^2 + u v';  an 8-bit state's v is its root's square, one more: 3 u
    p'   update = rate m' / (r root + eps): rate u, root 2 u, r half of v's relative error and u, the sum u, the reciprocal 2 u (1 ulp),
         two products: 10 u |update| + |update| (dm / |m'| + dv / 2 v');  p keep: keep and the product, 2 u |p|; the sum u |p'|.
A bf16 parameter is half a step of its type off its master, or off that."""
import math

import numpy as np
import pytest

from gpu_util import host, say, torch
from oracle import adamw as oracle
from test_gpu_norm import half_step, near

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


class Set:
    """Tensors of an optimizer cut out of buffers of their kind, each `shift` elements from the start of its own: every
    alignment occurs.  Buffers hold 7 (77 for codes) between the tensors."""

    def __init__(self, sizes, param="fp32", grad="fp32", eight=False, master=False, shift=0, seed=0, codes_of=None):
        t = torch()
        g = t.Generator(device="cuda")
        g.manual_seed(seed)
        dt = {"fp32": t.float32, "bf16": t.bfloat16}
        self.buffers, self.sizes, self.eight = [], list(sizes), eight

        def cut(make, dtype, fill, each=lambda n: n):
            room = [each(n) + 13 for n in sizes]
            flat = t.full((sum(room) + 64,), fill, device="cuda", dtype=dtype)
            out, at = [], shift
            for i, (n, r) in enumerate(zip(sizes, room)):
                v = flat[at: at + each(n)]
                v.copy_(make(each(n)))
                out.append(v)
                at += r
            self.buffers.append((flat, fill, out))
            return out
        r = lambda n: t.randn(n, generator=g, device="cuda")
        self.grads = cut(lambda n: r(n) * 1e-3, dt[grad], 7)
        values = [r(n) * 0.02 for n in sizes]
        it = iter(values)
        self.params = cut(lambda n: next(it), dt[param], 7)
        it = iter(values)
        self.masters = cut(lambda n: next(it), t.float32, 7) if master else None
        if eight:
            ints = lambda n, lo, hi: t.randint(lo, hi, (n,), generator=g, device="cuda").to(t.uint8)
            # every code but NaN's two; roots are not negative
            self.avg = cut(lambda n: ints(n, 0, 127) | ints(n, 0, 2) * 128, t.uint8, 77)
            self.sq = cut(lambda n: ints(n, 0, 127), t.uint8, 77)
            blocks = lambda n: -(-n // 128)
            self.avg_scale = cut(lambda n: (r(n).abs() + 0.1) * 1e-6, t.float32, 7, blocks)
            self.sq_scale = cut(lambda n: (r(n).abs() + 0.1) * 3e-6, t.float32, 7, blocks)
        else:
            self.avg = cut(lambda n: r(n) * 3e-4, t.float32, 7)
            self.sq = cut(lambda n: (r(n) * 1e-3).square(), t.float32, 7)
            self.avg_scale = self.sq_scale = None

    def step(self, P, step, **k):
        P.puro_adamw(self.params, self.grads, self.avg, self.sq, step, masters=self.masters, avg_scales=self.avg_scale,
                     sq_scales=self.sq_scale, **{**HYPER, **k})

    def gaps_untouched(self):
        for flat, fill, parts in self.buffers:
            copy = flat.clone()
            base = flat.storage_offset()
            for v in parts:
                copy[v.storage_offset() - base:][: v.numel()] = fill
            assert (copy == fill).all()

    def copies(self):
        c = lambda v: None if v is None else [x.clone() for x in v]
        return [c(v) for v in (self.params, self.masters, self.avg, self.sq, self.avg_scale, self.sq_scale)]


def expected(s, before, i, step, coef, h):
    """Tensor i's (m', v', p') in 64 bits, and their bounds."""
    params, masters, avg, sq, sa, sr = before
    d = lambda v: v[i].double()
    if s.eight:
        m, r = (torch().from_numpy(oracle.decode(host(c[i]), host(f[i]))).cuda().double() for c, f in ((avg, sa), (sq, sr)))
        v = r * r
    else:
        m, v = d(avg), d(sq)
    g = d(s.grads) * coef
    c1, c2 = 1 - h["beta1"], 1 - h["beta2"]
    m1 = h["beta1"] * m + c1 * g
    v1 = h["beta2"] * v + c2 * g * g
    dm = 2 * U * (h["beta1"] * m).abs() + 7 * U * (c1 * g).abs() + U * m1.abs()
    dv = 3 * U * h["beta2"] * v + 13 * U * c2 * g * g + U * v1
    p = d(masters if masters is not None else params)
    den = (v1 / (1 - h["beta2"] ** step)).sqrt() + h["eps"]
    update = h["lr"] / (1 - h["beta1"] ** step) * m1 / den
    p1 = p * (1 - h["lr"] * h["weight_decay"]) - update
    dp = 10 * U * update.abs() + (update / m1).abs().nan_to_num(0) * dm + update.abs() * (dv / (2 * v1)).nan_to_num(0)
    return m1, v1, p1, dm + 1e-45, dv + 1e-44, dp + 2 * U * p.abs() + U * p1.abs()


SIZES = [[1], [0], [3, 0, 5], [7, 8, 9], [127, 128, 129], [4096], [4097, 4095, 1], [100003], [1 << 20, 17, 4096], [5] * 200, [2048 * 512, 2047]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("param,grad,master", [("fp32", "fp32", False), ("fp32", "bf16", False), ("bf16", "fp32", True),
                                               ("bf16", "bf16", True), ("bf16", "bf16", False)])
@pytest.mark.parametrize("eight", [False, True])
def test_step(P, sizes, param, grad, master, eight):
    t = torch()
    for shift, clip, step in ((0, None, 1), (1, 0.5, 7), (3, 1e9, 5000)):
        say(f"[adamw] {sizes[:4]} {param} {grad} master {master} eight {eight} shift {shift} step {step}")
        s = Set(sizes, param, grad, eight, master, shift, len(sizes) + shift)
        before = s.copies()
        how, coef = {}, 1.0
        if clip is not None:
            norm = P.puro_grad_norm(s.grads)
            how, coef = dict(norm=norm, max_norm=clip * float(norm)), min(1.0, clip * float(norm) / (float(norm) + 1e-6))
        s.step(P, step, seed=99 + step, **how)
        s.gaps_untouched()
        for i, n in enumerate(sizes):
            m1, v1, p1, dm, dv, dp = expected(s, before, i, step, coef, HYPER)
            held = s.masters[i] if master else s.params[i]
            near(held, p1, dp + (half_step(p1.abs() + dp, held.dtype) if held.dtype == t.bfloat16 else 0), "param")
            if master:
                assert t.equal(s.params[i], held.bfloat16())
            if not eight:
                near(s.avg[i], m1, dm, "exp_avg")
                near(s.sq[i], v1, dv, "exp_avg_sq")
            elif n:
                c = 1.0
                if clip is not None:
                    f = np.float32
                    c = min(f(1), f(how["max_norm"]) / (f(float(norm)) + f(1e-6)))
                qa, qr, sa, sr, _, _ = oracle.step8(host(s.grads[i]).astype(np.float32), host(before[2][i]), host(before[3][i]),
                                                    host(before[4][i]), host(before[5][i]), HYPER["beta1"], HYPER["beta2"],
                                                    99 + step, step, i, c)
                assert np.array_equal(host(s.avg_scale[i]), sa) and np.array_equal(host(s.sq_scale[i]), sr)
                assert np.array_equal(host(s.avg[i]), qa) and np.array_equal(host(s.sq[i]), qr)


def test_first_steps_from_zero(P):
    """Ten steps from states of zero against the formula in 64 bits: each step adds at most its own bound to the parameters'
    error, and the states' relative errors grow by at most their own bound a step (their factors are below 1)."""
    t = torch()
    for eps in (1e-8, 0.0):
        s = Set([1000], shift=1)
        s.avg[0].zero_(), s.sq[0].zero_()
        p, m, v = s.params[0].double(), t.zeros(1000, dtype=t.float64, device="cuda"), t.zeros(1000, dtype=t.float64, device="cuda")
        h = {**HYPER, "eps": eps}
        off = 0.0
        for k in range(1, 11):
            s.grads[0].normal_(0, 1e-3)
            g = s.grads[0].double()
            m, v = 0.9 * m + 0.1 * g, 0.95 * v + 0.05 * g * g
            update = h["lr"] / (1 - 0.9 ** k) * m / ((v / (1 - 0.95 ** k)).sqrt() + eps)
            p = p * (1 - h["lr"] * 0.1) - update
            # m's terms may cancel: their error is that of the gradients' sizes so far, below 8 u of the largest a step
            off = off + 10 * U * update.abs() + 8 * k * U * h["lr"] / (1 - 0.9 ** k) * 5e-3 / (v / (1 - 0.95 ** k)).sqrt() \
                + 16 * k * U * update.abs() + 3 * U * (p.abs() + update.abs())
            s.step(P, k, eps=eps)
            near(s.params[0], p, off, f"step {k}")


def test_hyperparameters(P):
    t = torch()
    for h in (dict(beta1=0.0), dict(beta2=0.0), dict(lr=0.0), dict(weight_decay=0.0), dict(lr=-1e-3), dict(eps=1.0), dict(beta2=0.9999)):
        s = Set([5000], shift=2)
        before = s.copies()
        s.step(P, 3, **h)
        m1, v1, p1, dm, dv, dp = expected(s, before, 0, 3, 1.0, {**HYPER, **h})
        near(s.params[0], p1, dp, h)
        near(s.avg[0], m1, dm, h)
        near(s.sq[0], v1, dv, h)


def test_step_and_rate_on_the_device(P):
    """The same bits as given from the host, for every kind of states."""
    t = torch()
    for eight in (False, True):
        a, b, c = (Set([3000, 77], eight=eight, shift=1, seed=5) for _ in range(3))
        lr = float(np.float32(1e-3))
        a.step(P, 123456, lr=lr, seed=7)
        b.step(P, t.tensor([123456], device="cuda"), lr=t.tensor(1e-3, device="cuda"), seed=7)
        c.step(P, 123456, lr=t.tensor(1e-3, device="cuda"), seed=7)
        for x, y, z in zip(a.copies(), b.copies(), c.copies()):
            assert x is None or all(t.equal(p, q) and t.equal(p, r) for p, q, r in zip(x, y, z))


def test_random_words_follow_seed_step_and_place(P):
    t = torch()

    def alike(n):
        """n tensors with the values of the first of a list of one."""
        one, s = Set([1000], eight=True, seed=3), Set([1000] * n, eight=True, seed=3)
        for v, w in zip((s.grads, s.avg, s.sq, s.avg_scale, s.sq_scale), (one.grads, one.avg, one.sq, one.avg_scale, one.sq_scale)):
            for x in v:
                x.copy_(w[0])
        return s

    def codes(seed=1, step=2, n=1):
        s = alike(n)
        s.step(P, step, seed=seed)
        return [x.clone() for x in s.avg]
    base = codes()
    assert t.equal(codes()[0], base[0]) and not t.equal(codes(seed=2)[0], base[0]) and not t.equal(codes(step=3)[0], base[0])
    assert not t.equal(codes(seed=1 + 2 ** 32)[0], base[0])
    two = codes(n=2)
    assert t.equal(two[0], base[0]) and not t.equal(two[1], base[0])
    # an empty tensor in front, and tensors of fp32 states in between, keep their places in the list
    s = alike(2)
    z = lambda n, d=t.float32: t.zeros(n, device="cuda", dtype=d)
    for x in (s.grads, s.avg, s.sq, s.avg_scale, s.sq_scale):
        x[1].copy_(x[0])
    P.puro_adamw([s.params[0], z(5), s.params[1]], [s.grads[0], z(5), s.grads[1]], [s.avg[0], z(5), s.avg[1]],
                 [s.sq[0], z(5), s.sq[1]], 2, avg_scales=[s.avg_scale[0], None, s.avg_scale[1]],
                 sq_scales=[s.sq_scale[0], None, s.sq_scale[1]], seed=1, **HYPER)
    assert t.equal(s.avg[0], base[0]) and not t.equal(s.avg[1], base[0]) and not t.equal(s.avg[1], two[1])


def test_non_finite_gradients(P):
    t = torch()
    for eight in (False, True):
        s, clean = Set([1000], eight=eight), Set([1000], eight=eight)
        s.grads[0][5], s.grads[0][300] = float("nan"), float("inf")
        clean.step(P, 4)
        s.step(P, 4)
        p, q = s.params[0], clean.params[0]
        assert p[5].isnan() and p[300].isnan()
        keep = t.ones(1000, dtype=t.bool, device="cuda")
        keep[5] = keep[300] = False
        assert t.equal(p[keep], q[keep])
        if eight:
            assert (s.avg[0][5] & 0x7F) == 0x7F and (s.sq[0][5] & 0x7F) == 0x7F and (s.avg[0][300] & 0x7F) == 0x7F
            other = [i for i in range(1000) if i != 5 and not 256 <= i < 384]
            # (where the NaN stood, the clean one's value may have set the scale of its block)
            far = [i for i in other if i >= 128]
            assert t.equal(s.avg[0][far], clean.avg[0][far]) and t.equal(s.sq[0][far], clean.sq[0][far])
            s.grads[0].zero_()
            s.step(P, 5)
            assert p[256:384].isnan().all() and p[5].isnan() and p[384:].isfinite().all() and p[6:256].isfinite().all()
        else:
            assert s.avg[0][5].isnan() and s.sq[0][5].isnan() and s.sq[0][300].isinf()
    s = Set([1000])
    s.step(P, 1, norm=t.tensor(float("nan"), device="cuda"))
    assert s.params[0].isnan().all()
    s, z = Set([1000]), Set([1000])
    s.step(P, 1, norm=t.tensor(float("inf"), device="cuda"))           # a factor of 0: as gradients of zero
    z.grads[0].zero_()
    z.step(P, 1)
    assert t.equal(s.params[0], z.params[0])


def test_eight_bit_states_keep_up_with_the_gradients(P):
    """Roots that start 16 times too high come down to gradients of one size with beta2 = 0.999, where each step moves them by
    a hundredth of a code.  From 16 |g| the decay alone takes 2 ln(16) / 0.001 = 5500 steps; after 12000 steps v / g^2 is 1 +
    256 e^-12 = 1.002.  The root's deviation from the walk of its rounding is sqrt(step / 2 / 2) at most, 18% (a code's
    step is at most 1/8): mean of n = 65536 independent ones within 6 of their deviations, and its bias below
    half its variance, 2%."""
    t = torch()
    n, size = 65536, 1e-3
    s = Set([n], eight=True)
    s.sq[0].fill_(0x7E)
    s.sq_scale[0].fill_(16 * size / 448)
    s.avg[0].zero_()
    for k in range(1, 12001):
        if k % 100 == 1:
            s.grads[0].copy_(t.where(t.rand(n, device="cuda") < 0.5, -size, size))
        s.step(P, k, beta2=0.999, seed=5)
    root = t.from_numpy(oracle.decode(host(s.sq[0]), host(s.sq_scale[0]))).double() / size
    say(f"[adamw] root / |g|: mean {float(root.mean()):.4f}, deviation {float(root.std()):.4f}")
    assert float(root.std()) <= 0.18 and abs(float(root.mean()) - 1.001) <= 0.02 + 6 * 0.18 / math.sqrt(n)


@pytest.mark.parametrize("exponent", [-149, -126, -100, -60, -49, -48, -47, -30, -1, 20, 40, 62])
def test_states_of_every_size(P, exponent):
    """Gradients and states about 2^exponent, of many sizes within a block, zeros among them, down to subnormal numbers and squares
    that vanish or overflow: 8-bit states as the oracle's, to the bit; a block of one size beside them."""
    t = torch()
    n = 128 * 40 + 77
    s = Set([n], eight=True, seed=exponent & 255)
    g = t.Generator(device="cuda")
    g.manual_seed(5)
    size = t.exp2(exponent + 12 * t.rand(n, generator=g, device="cuda", dtype=t.float64))
    size[::7] = 0
    size[1280:1408] = 2.0 ** exponent
    size[2560:3000] = 0
    s.grads[0].copy_(size * t.randn(n, generator=g, device="cuda"))
    for scale, part in ((s.avg_scale[0], 0.1), (s.sq_scale[0], 0.3)):
        scale.copy_(t.full_like(scale, 1.0).double() * 2.0 ** max(exponent, -140) * part / 448)
    s.avg[0][2560:3000], s.sq[0][2560:2800] = 0, 0
    before = s.copies()
    s.step(P, 3, seed=8)
    with np.errstate(over="ignore", invalid="ignore"):
        qa, qr, sa, sr, _, _ = oracle.step8(host(s.grads[0]), *(host(before[k][0]) for k in (2, 3, 4, 5)), HYPER["beta1"],
                                            HYPER["beta2"], 8, 3, 0)
    assert np.array_equal(host(s.avg_scale[0]), sa) and np.array_equal(host(s.sq_scale[0]), sr)
    for got, want in ((host(s.avg[0]), qa), (host(s.sq[0]), qr)):        # (NaN has two codes, and zero's sign is none's)
        either = np.isin(want & 0x7F, (0, 0x7F))
        assert np.array_equal(got & 0x7F, want & 0x7F) and np.array_equal(got[~either], want[~either])


def test_roots_of_every_gradient(P):
    """The roots of v' = g g (beta2 = 0) for every mantissa of g, a block of 128 alike for each: a block's scale is its root times
    1 / 448 in fp32, and shows every bit of the root; of 8192 gradients beside it, at other exponents too."""
    t = torch()
    n = 1 << 20
    inv = t.tensor(float(np.float32(1) / np.float32(448)), device="cuda")
    p, m, v = (t.zeros(128 * n, dtype=d, device="cuda") for d in (t.bfloat16, t.uint8, t.uint8))
    sm, sv = t.zeros(n, device="cuda"), t.zeros(n, device="cuda")
    for first in range(0, 1 << 23, n):
        g = (t.arange(n, device="cuda", dtype=t.int32) + (0x3F800000 + first)).view(t.float32)
        if first == 0:
            g[:8192] = t.exp2(t.linspace(-47, 60, 8192, device="cuda"))
        P.puro_adamw([p], [g.repeat_interleave(128)], [m], [v], 1, 0.0, beta2=0.0, avg_scales=[sm], sq_scales=[sv])
        root = (g * g).double().sqrt().float()               # (53 bits are enough for the one rounding that counts)
        assert t.equal(sv, root * inv), first
        # 448, or, where three roundings left up to 3 u of it off and the chance is 0 of 65536, the code below: a binomial
        # variable of 2^27 draws with a mean of at most 2048 and a deviation of 45.3, six of them
        low = v == 0x7D
        assert ((v == 0x7E) | low).all() and int(low.sum()) <= 2048 + 6 * 45.3


def test_layouts(P):
    """Matrices dense in another order of their dimensions, with everything that goes with them in the same one."""
    t = torch()
    make = lambda d=t.float32: (t.randn((40, 24), device="cuda") * 1e-2).to(d)
    p, g, m, v = make(), make(), make(), make().square()
    flat = [x.clone() for x in (p, g, m, v)]
    turned = [x.t().contiguous().t() for x in (p, g, m, v)]
    P.puro_adamw([flat[0]], [flat[1]], [flat[2]], [flat[3]], 3, **HYPER)
    P.puro_adamw([turned[0]], [turned[1]], [turned[2]], [turned[3]], 3, **HYPER)
    for a, b in zip(flat, turned):
        assert t.equal(a, b)
    with pytest.raises(ValueError):
        P.puro_adamw([flat[0]], [turned[1]], [flat[2]], [flat[3]], 3, **HYPER)


def test_streams_graphs_and_versions(P):
    """A captured step reads its step number and rate at every replay; every replay is the eager step."""
    t = torch()
    for eight in (False, True):
        eager, graph, side = (Set([5000, 130, 1], eight=eight, seed=2) for _ in range(3))
        step, lr = t.ones(1, dtype=t.int64, device="cuda"), t.full((), 1e-3, device="cuda")
        norm = t.zeros((), device="cuda")
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            P.puro_grad_norm(graph.grads, norm=norm)
            graph.step(P, step, lr=lr, norm=norm, max_norm=0.01, seed=11)
        stream = t.cuda.Stream()
        stream.wait_stream(t.cuda.current_stream())
        for k in range(1, 5):
            for a, b, c in zip(eager.grads, graph.grads, side.grads):
                a.normal_(0, 1e-3)
                b.copy_(a)
                c.copy_(a)
            step.fill_(k)
            lr.fill_(1e-3 / k)
            g.replay()
            n = P.puro_grad_norm(eager.grads)
            eager.step(P, k, lr=float(np.float32(1e-3 / k)), norm=n, max_norm=0.01, seed=11)
            stream.wait_stream(t.cuda.current_stream())
            side.step(P, k, lr=float(np.float32(1e-3 / k)), norm=n, max_norm=0.01, seed=11, stream=stream if k % 2 else stream.cuda_stream)
            t.cuda.synchronize()
            for x, y, z in zip(eager.copies(), graph.copies(), side.copies()):
                assert x is None or all(t.equal(p, q) and t.equal(p, r) for p, q, r in zip(x, y, z)), (eight, k)
        before = [v._version for v in eager.params + eager.avg + eager.sq]
        eager.step(P, 9)
        assert all(v._version > b for v, b in zip(eager.params + eager.avg + eager.sq, before))


def test_more_than_32_bits_of_elements(P):
    """2^31 elements and some: the ends as by themselves (in blocks and groups of their own place, so with fp32 states and
    with 8-bit ones whose random words are the oracle's)."""
    t = torch()
    n = (1 << 31) + 8 * 16 + 5
    say("[adamw, large]")
    h = dict(HYPER)
    p, g = t.full((n,), 0.5, dtype=t.bfloat16, device="cuda"), t.full((n,), 1e-3, dtype=t.bfloat16, device="cuda")
    m, v = t.zeros(n, dtype=t.uint8, device="cuda"), t.zeros(n, dtype=t.uint8, device="cuda")
    sm, sv = (t.zeros(-(-n // 128), device="cuda") for _ in range(2))
    first = (1 << 31) - 1024
    g[first:] = (t.randn(n - first, device="cuda") * 1e-3).bfloat16()
    grad = host(g[first:]).astype(np.float32)
    P.puro_adamw([p], [g], [m], [v], 3, avg_scales=[sm], sq_scales=[sv], seed=4, **h)
    zero = np.zeros(n - first, np.uint8)
    m1, v1 = oracle.states(grad, zero.astype(np.float32), zero.astype(np.float32), 0.9, 0.95)
    word = oracle.random_words(4, 3, 0, n - first, first)
    qa, sa = oracle.encode(m1, word & np.uint64(0xFFFF), False)
    qr, sr = oracle.encode(np.sqrt(v1), word >> np.uint64(16), True)
    assert np.array_equal(host(m[first:]), qa) and np.array_equal(host(v[first:]), qr)
    assert np.array_equal(host(sm[first // 128:]), sa) and np.array_equal(host(sv[first // 128:]), sr)
    tail = [p[first:].clone(), g[first:].clone()]
    del m, v, sm, sv
    m, v = (t.zeros(n, device="cuda") for _ in range(2))
    P.puro_adamw([p], [g], [m], [v], 3, **h)
    a, b = (t.zeros(n - first, device="cuda") for _ in range(2))
    P.puro_adamw([tail[0]], [tail[1]], [a], [b], 3, **h)
    assert t.equal(p[first:], tail[0]) and t.equal(m[first:], a) and t.equal(v[first:], b)


def test_refusals(P):
    t = torch()
    f = lambda n=300, d=t.float32: t.zeros(n, device="cuda", dtype=d)
    u8 = lambda: f(300, t.uint8)

    def refused(error, *a, **k):
        with pytest.raises(error):
            P.puro_adamw(*a, **{**HYPER, **k})
    ok = [[f()], [f()], [f()], [f()]]
    refused(TypeError, None, *ok[1:], 1)
    refused(TypeError, ok[0], None, *ok[2:], 1)
    refused(ValueError, ok[0], [], *ok[2:], 1)
    refused(ValueError, ok[0], [f(299)], *ok[2:], 1)
    refused(TypeError, [f(300, t.float16)], *ok[1:], 1)
    refused(TypeError, ok[0], ok[1], [u8()], [u8()], 1)
    refused(TypeError, *ok, 1, avg_scales=[f(3)], sq_scales=[f(3)])
    refused(ValueError, ok[0], ok[1], [u8()], [u8()], 1, avg_scales=[f(2)], sq_scales=[f(3)])
    refused(ValueError, ok[0], ok[1], [u8()], [u8()], 1, avg_scales=[f(3)])
    refused(ValueError, ok[0], ok[1], [u8()], [u8()], 1, avg_scales=[f(3)], sq_scales=[None])
    refused(ValueError, *ok, 1, masters=[f()])
    refused(ValueError, [f().cpu()], *ok[1:], 1)
    refused(TypeError, *ok, "1")
    refused(TypeError, *ok, t.ones(1, device="cuda"))
    refused(TypeError, *ok, 1, lr=t.ones(1, device="cuda").double())
    refused(ValueError, *ok, t.ones(2, dtype=t.int64, device="cuda"))
    refused(ValueError, *ok, 1, seed=-1)
    refused(TypeError, *ok, 1, seed=1.5)
    for bad in (dict(beta1=1.0), dict(beta2=-0.1), dict(lr=float("nan")), dict(eps=-1e-8), dict(weight_decay=float("inf")),
                dict(norm=f(1), max_norm=-1.0), dict(norm=f(1), max_norm=float("nan"))):
        refused(P.PuroError, *ok, 1, **bad)
    refused(P.PuroError, *ok, 0)
    one = f()
    refused(P.PuroError, [one], [one], [f()], [f()], 1)                # a gradient that is the parameter
    refused(P.PuroError, [one, one], [f(), f()], [f(), f()], [f(), f()], 1)
    refused(P.PuroError, [f()], [f()], [one], [one], 1)
    refused(P.PuroError, [one], [f()], [f()], [f()], 1, norm=one[:1])
    refused(P.PuroError, [f()], [f()], [f()], [one], 1, lr=one[:1])
    g = f()
    P.puro_adamw([f(), f()], [g, g], [f(), f()], [f(), f()], 1, **HYPER)     # a gradient may serve two parameters
    P.puro_adamw([], [], [], [], 1, **HYPER)
