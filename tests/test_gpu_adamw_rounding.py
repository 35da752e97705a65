"""GPU tests of the short sequences of the AdamW step: a root and a reciprocal, each an instruction's value with one correction, are
correctly rounded for every mantissa.  What a wrong one would change is shown to be seen: the references of two neighbouring
roots differ, and a multiplier one unit off, either way, changes a code of every block.

The references are roots and quotients in 64 bits, rounded: 53 bits are enough (2 * 24 + 2) for the one rounding that counts."""
import numpy as np
import pytest

from gpu_util import host, say, torch
from oracle import adamw as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def floats(first, n, dtype=None):
    """n neighbouring fp32 numbers, from that of the bits `first`."""
    t = torch()
    return (t.arange(n, device="cuda", dtype=t.int32) + first).view(t.float32)


ONE, HALF_STEP = 0x3F800000, 2.0 ** -24
# r + offset: just above 2 for some part of [1, 2), where neighbouring reciprocals lie further apart than fp32 numbers; a half step and
# one and a half of r's, so that the sum, whose steps are twice r's, keeps each pair of neighbours apart in one of the two
OFFSETS = [0.0] + [b + k * HALF_STEP for b in (0.59375, 0.40625, 0.203125) for k in (1, 3)]


@pytest.mark.parametrize("k", [0, -48, 62])
def test_roots_of_every_value(P, k):
    """v over [1, 4) times 4^k, every fp32 number: from 2^-96, the least that takes the short root, to 2^126.  The states are given
    as they are (gradients of zero, betas that round to 1), so that v' = v and p' = -1 / (root + eps), the reciprocal by its
    instruction.  It is the same as from v2 = r r (rounded) for the root r that v ought to have: sqrt(v2) is at most
    0.354 of a unit off r, so that no root of it that is right to 2^-19 before its last rounding can be another."""
    t = torch()
    n = 1 << 23
    r = floats(ONE, n)                                    # every root
    v = floats(ONE, 2 * n)                                # [1, 4): two binades of n
    want = v.double().sqrt().float()
    at = want.view(t.int32).long() - ONE
    assert int(at.min()) == 0 and int(at.max()) == n - 1
    assert ((r * r).double().sqrt() - r.double()).abs().max() <= 0.36 * 2.0 ** -23
    apart = t.zeros(n - 1, dtype=t.bool, device="cuda")

    def updates(v, eps):
        p, g, m = t.zeros_like(v), t.zeros_like(v), t.ones_like(v)
        w = v * 4.0 ** k
        kept = w.clone()
        P.puro_adamw([p], [g], [m], [w], 1 << 40, 1.0, 1 - 2.0 ** -30, 1 - 2.0 ** -30, eps * 2.0 ** k, 0.0)
        assert t.equal(w, kept) and (m == 1).all()
        return p
    for eps in OFFSETS:
        say(f"[adamw, roots] 4^{k}, eps {eps}")
        ref = updates(r * r, eps)
        apart |= ref[1:] != ref[:-1]
        got = updates(v, eps)
        assert t.equal(got, ref[at]), int((got != ref[at]).sum())
    assert apart.all(), int((~apart).sum())


def test_roots_of_every_value_in_the_scales(P):
    """The 8-bit step's roots of every v of [1, 4), a block of 128 alike for each: v' = A + c2 g g with A from the old root and g
    chosen for it; a block's scale is its root times 1 / 448 in fp32."""
    t = torch()
    n = 1 << 19
    inv = t.tensor(float(np.float32(1) / np.float32(448)), device="cuda")
    p, m, code = (t.zeros(128 * n, dtype=d, device="cuda") for d in (t.bfloat16, t.uint8, t.uint8))
    sm, sv = t.zeros(n, device="cuda"), t.zeros(n, device="cuda")
    for first in range(0, 1 << 24, n):
        v = floats(ONE + first, n)
        start = float(v[0])
        old = float(np.float32(np.sqrt(2 * start)))       # half its square is at most v, or a little above it
        while np.float32(0.5) * (np.float32(old) * np.float32(old)) > np.float32(start):
            old = float(np.nextafter(np.float32(old), np.float32(0)))
        a = t.tensor(old, device="cuda")
        a = 0.5 * (a * a)
        g = (2 * (v.double() - a.double())).sqrt().float()
        assert t.equal(a + 0.5 * g * g, v), first         # (each operation by itself, as the step's)
        code.fill_(0x38)                                  # 1.0
        m.zero_(), sm.zero_(), sv.fill_(old)
        P.puro_adamw([p], [g.repeat_interleave(128)], [m], [code], 1, 0.0, beta2=0.5, avg_scales=[sm], sq_scales=[sv])
        assert t.equal(sv, v.double().sqrt().float() * inv), first


def code_of(y, chance):
    """E4M3 codes of y (0.5 to 448) after its mantissa is cut behind 16 random bits."""
    t = torch()
    cut = ((y.view(t.int32) + (chance << 4)) & -0x100000).view(t.float32)
    return cut.to(t.float8_e4m3fn).view(t.uint8)


@pytest.mark.parametrize("k", [0, -40, 60])
def test_multipliers_of_every_largest_value(P, k):
    """Blocks whose largest value a runs over every mantissa (k = 0; else a part, the all-ones one among them): the codes of values
    that lie where their random bits just carry into the code, or just do not."""
    t = torch()
    n = 1 << 17                                            # blocks of a call
    chance = t.from_numpy((oracle.random_words(5, 9, 0, 128 * n) & np.uint64(0xFFFF)).astype(np.int32)).cuda().view(n, 128)
    g = t.Generator(device="cuda")
    g.manual_seed(1)
    one = t.tensor(float(np.float32(1) / np.float32(448)), device="cuda")
    p = t.zeros(128 * n, dtype=t.bfloat16, device="cuda")
    f = t.float32
    for first in range(0, 1 << 23, n) if k == 0 else (0, (1 << 22) + 12345, (1 << 23) - n):
        a = floats(ONE + first, n) * 2.0 ** k
        mult = 448.0 * (1.0 / a.double()).float()          # the definition: the reciprocal rounded, then the product
        units = mult.view(t.int32)
        # a border of codes that y meets: 1 to 256, less what the random bits add
        border = t.randint(0x3F8, 0x438, (n, 128), generator=g, device="cuda", dtype=t.int32) << 20
        least = (border - (chance << 4)).view(f)           # the least y that is carried over it
        x = (least.double() / mult.double()[:, None]).float()
        y = lambda x, by=0: x * (units + by).view(f)[:, None]
        near = t.stack([(x.view(t.int32) + d).view(f) for d in (-2, -1, 0, 1, 2)])
        over = t.stack([y(v) >= least for v in near])
        assert over[-1].all() and not over[0].any()
        count = (~over).sum(0)                             # places below the border
        above, below = near.gather(0, count[None])[0], near.gather(0, count[None] - 1)[0]
        x = t.where(t.arange(128, device="cuda") % 2 == 0, above, below)
        x[:, 0] = a
        assert (x.abs().amax(1) == a).all()
        want = code_of(y(x), chance)
        for by in (-1, 1):
            assert (code_of(y(x, by), chance) != want).any(1).all(), (first, by)
        m, v = (t.zeros(128 * n, dtype=t.uint8, device="cuda") for _ in range(2))
        sm, sv = t.zeros(n, device="cuda"), t.zeros(n, device="cuda")
        P.puro_adamw([p], [x.view(-1)], [m], [v], 9, 0.0, 0.0, 0.0, avg_scales=[sm], sq_scales=[sv], seed=5)
        assert t.equal(sm, a * one) and t.equal(m.view(n, 128), want), first
    say(f"[adamw, multipliers] 2^{k}")
