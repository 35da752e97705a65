"""GPU tests of clipping over the views of one flat bucket: neighbours share 16-byte vectors, which are read and written
element by element at a tensor's ends.

Tolerance, with u = 2^-24: norm 2 u, coefficient 4 u, product 1 u, and half a step of bf16 (2^-8)."""
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


SIZES = {"short": [1, 2, 3, 5, 7, 1, 1, 9, 4, 8, 16, 31, 1, 6], "mixed": [4097, 1, 8191, 3, 100003, 7, 12288, 5, 1, 2047],
         "many": [1 + 37 * i % 61 for i in range(400)]}


@pytest.mark.parametrize("sizes", SIZES.values(), ids=SIZES.keys())
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("start", [0, 1, 5])
def test_views_of_one_bucket(P, sizes, dtype, start):
    t = torch()
    dt = getattr(t, dtype)
    n = sum(sizes)
    g = t.Generator(device="cuda")
    g.manual_seed(n + start)
    flat = (t.randn(n + 32, generator=g, device="cuda") * 1e-2).to(dt)
    views = lambda b: list(b[start:start + n].split(sizes))
    ref = flat[start:start + n].double()
    norm64 = math.sqrt(float(ref.square().sum()))
    for max_norm in (0.4 * norm64, 2 * norm64 + 1):
        say(f"[bucket] {len(sizes)} tensors, {n} elements {dtype} from {start}, bound {max_norm:.3g}")
        want = ref * min(1.0, max_norm / (norm64 + 1e-6))
        bound = want.abs() * (7 * U + (2.0 ** -8 * (1 + 2.0 ** -7) if dtype == "bfloat16" else 0.0))
        mine, other = flat.clone(), t.full((n + 32,), 9.0, device="cuda", dtype=dt)
        shifted = t.full((n + 33,), 9.0, device="cuda", dtype=dt)
        norm, _ = P.puro_clip_grad_norm(views(mine), max_norm)
        P.puro_clip_grad_norm(views(flat), max_norm, outs=views(other))
        P.puro_clip_grad_norm(views(flat), max_norm, outs=views(shifted[1:]))        # outputs at another alignment
        assert abs(float(norm) - norm64) <= 2 * U * norm64
        assert ((mine[start:start + n].double() - want).abs() <= bound).all()
        assert t.equal(mine[:start], flat[:start]) and t.equal(mine[start + n:], flat[start + n:])
        assert t.equal(other[start:start + n], mine[start:start + n]) and t.equal(shifted[start + 1:start + 1 + n], mine[start:start + n])
        for b, lo in ((other, start), (shifted, start + 1)):
            assert (b[:lo] == 9).all() and (b[lo + n:] == 9).all()
        # every second view alone: what lies between stays
        odd = flat.clone()
        P.puro_clip_grad_norm(views(odd)[1::2], 0.0)
        for k, (a, b) in enumerate(zip(views(odd), views(flat))):
            assert (a == 0).all() if k % 2 else t.equal(a, b)
