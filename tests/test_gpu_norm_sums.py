"""GPU tests of the weight's and bias's gradient of the norm over many rows: the error does not grow with their number.

Tolerance, with u = 2^-24: a thread adds at most 64 rows in order and at most 64 such sums, a workgroup up to 32 of those,
a run of workgroups 16, and 16 runs are joined; each term has two roundings before its addition, and 64-bit sums between
16 workgroups and the next are rounded once: (64 + 64 + 32 + 16 + 16 + 3) u sum|terms|.  (The longest inputs have more than 256 workgroups.)"""
import pytest

from gpu_util import say, torch

pytestmark = pytest.mark.gpu
BOUND = (64 + 64 + 32 + 16 + 16 + 3) * 2.0 ** -24


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


@pytest.mark.parametrize("T,C", [(262144, 4104), (262144 * 32, 8), (1 << 20, 2000), ((1 << 25) + 5, 8)])
def test_terms_that_round_one_way(P, T, C):
    """Terms of 1 + 2^-15 - 2^-23: between 512 and 1024 a sum's step is 2^-14, and each addition there loses nearly half
    of one.  512 such additions in order are 256 u off."""
    t = torch()
    say(f"[norm sums] {T}x{C}")
    term = 1 + 2.0 ** -15 - 2.0 ** -23
    x = t.ones((T, C), device="cuda")
    dy = t.full((T, C), term, device="cuda")
    w, mean, rstd = t.ones(C, device="cuda"), t.zeros(T, device="cuda"), t.ones(T, device="cuda")
    _, dw, db = P.puro_layer_norm_backward(dy, x, w, mean, rstd, dx=x)
    for got in (dw, db):
        assert float((got.double() / (T * term) - 1).abs().max()) <= BOUND
    _, dw, none = P.puro_layer_norm_backward(dy, t.ones_like(dy), w, None, rstd, kind=P.RMS_NORM, with_bias=False, dx=x)
    assert none is None and float((dw.double() / (T * term) - 1).abs().max()) <= BOUND


@pytest.mark.parametrize("T,C", [(262272, 8192), (70001, 4097), (1000003, 130), (40000, 16384), ((1 << 25) + 77, 3), ((1 << 22) + 9, 1030)])
def test_random_rows(P, T, C):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(T)
    say(f"[norm sums, random] {T}x{C}")
    x = t.randn((T, C), generator=g, device="cuda", dtype=t.bfloat16)
    dy = t.randn((T, C), generator=g, device="cuda", dtype=t.bfloat16)
    w = t.ones(C, device="cuda")
    _, mean, rstd = P.puro_layer_norm(x, w)
    _, dw, db = P.puro_layer_norm_backward(dy, x, w, mean, rstd)
    rw, rb, sw, sb = (t.zeros(C, dtype=t.float64, device="cuda") for _ in range(4))
    step = (1 << 26) // C
    for lo in range(0, T, step):
        part = slice(lo, lo + step)
        d = dy[part].double()
        v = d * ((x[part].double() - mean[part, None].double()) * rstd[part, None].double())
        rw += v.sum(0)
        rb += d.sum(0)
        sw += v.abs().sum(0)
        sb += d.abs().sum(0)
    assert ((dw.double() - rw).abs() <= BOUND * sw).all() and ((db.double() - rb).abs() <= BOUND * sb).all()
