"""GPU tests of the operators' `stream` argument given as a handle: the default stream's is 0."""
import pytest

from gpu_util import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def test_handle_of_the_default_stream(P):
    """Inputs whose producer is still pending on the default stream, and outputs used there: stream=0 orders both."""
    t = torch()
    assert t.cuda.current_stream().cuda_stream == 0
    v = t.randn((256, 512), device="cuda").bfloat16()
    w, wc = t.ones(512, device="cuda").bfloat16(), t.randn((256, 512), device="cuda").bfloat16()
    wq, ws, _, _ = P.puro_fp8_quant_w_128x128(wc)

    def step(x, stream):
        y, m, r = P.puro_layer_norm(x, w, stream=stream)
        q, s = P.puro_layer_norm_quant(x, w, stream=stream)
        dual = P.puro_layer_norm_quant_dual(x, w, stream=stream)
        back = P.puro_layer_norm_backward(y, x, w, m, r, stream=stream)
        rows = P.puro_gemm_rows(q, s, wq, ws, stream=stream)
        n, _ = P.puro_clip_grad_norm([y.clone()], 1.0, stream=stream)
        P.puro_scale_by_norm([rows], 1.0, P.puro_grad_norm([rows], stream=stream), stream=stream)
        return [y, m, r, q, s, *dual, *back, rows, n]

    want = [o.clone() for o in step(v, None)]
    t.cuda.synchronize()
    x = t.zeros_like(v)
    t.cuda.synchronize()
    t.cuda._sleep(20_000_000)                     # some 10 ms of the default stream
    x.copy_(v)
    got = [o.clone() for o in step(x, 0)]
    t.cuda.synchronize()
    for a, b in zip(got, want):
        assert t.equal(a, b)
