"""GPU tests of the norm's quantized forms: the codes are those of the tensor form's fp32 norm, exactly, so that rows far
from zero (constant ones, large offsets) keep what the tensor form keeps."""
import numpy as np
import pytest

from gpu_util import say, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def codes(y):
    """1x128 codes and scales of fp32 y [R, K], in fp32 steps on the CPU: maximum, two divisions, one product, one
    rounding to E4M3."""
    t = torch()
    R, K = y.shape
    v = y.cpu().numpy().reshape(R, K // 128, 128)
    amax = np.maximum(np.abs(v).max(2), np.float32(2.0 ** -96))
    s, r = (amax / np.float32(448)).astype(np.float32), (np.float32(448) / amax).astype(np.float32)
    q = t.from_numpy((v * r[:, :, None]).reshape(R, K)).to(t.float8_e4m3fn).view(t.uint8)
    return q.cuda(), t.from_numpy(np.ascontiguousarray(s.T)).cuda()


@pytest.mark.parametrize("C", [128, 640, 2048, 8192, 16384])
@pytest.mark.parametrize("xdtype", ["bfloat16", "float32"])
def test_codes_are_the_tensor_forms(P, C, xdtype):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(C)
    x = t.randn((128, C), generator=g, device="cuda") + 0.25
    for row, value in ((1, 30000.0), (2, 1000.0), (3, 7.5), (4, -0.3), (5, 0.0)):
        x[row] = value
    x[6] += 1e4
    x[7] = 3e4 + 128 * (x[7] > 0.25)                     # two neighbouring values of bf16
    x = x.to(getattr(t, xdtype))
    w = 1 + 0.3 * t.randn(C, generator=g, device="cuda")
    for kind, b in ((0, 0.2 * t.randn(C, generator=g, device="cuda")), (0, None), (1, None)):
        say(f"[norm codes] {C} {xdtype} kind {kind} bias {b is not None}")
        y, _, _ = P.puro_layer_norm(x.float(), w, b, kind=kind)
        want_q, want_s = codes(y)
        q, s = P.puro_layer_norm_quant(x, w, b, kind=kind)
        assert t.equal(s, want_s) and t.equal(q.view(t.float8_e4m3fn).float(), want_q.view(t.float8_e4m3fn).float())
        want_qT, want_sT = codes(y.t().contiguous())
        dq, ds, qT, sT, _, _ = P.puro_layer_norm_quant_dual(x, w, b, kind=kind)
        assert t.equal(dq, q) and t.equal(ds, s)
        assert t.equal(sT, want_sT) and t.equal(qT.view(t.float8_e4m3fn).float(), want_qT.view(t.float8_e4m3fn).float())


def test_constant_rows_leave_the_bias(P):
    """Rows of one power of two, whose sums are exact in any order: the difference from the mean is zero and the codes
    are the bias's."""
    t = torch()
    C = 2048
    x = t.full((128, C), 16384.0, device="cuda").bfloat16()
    w, b = t.ones(C, device="cuda"), 1e-3 * t.randn(C, device="cuda")
    want = codes(b.expand(128, C).contiguous())
    q, s = P.puro_layer_norm_quant(x, w, b)
    assert t.equal(q, want[0]) and t.equal(s, want[1])
    q, s = P.puro_layer_norm_quant(x, w)
    assert (q & 0x7F == 0).all() and (s == s[0, 0]).all()
