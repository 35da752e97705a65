"""GPU tests of a Rotary module whose first call on the GPU is made in inference mode, under a capture, or on another stream."""
import pytest

from gpu_util import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def test_training_after_a_first_call_in_inference_mode(P):
    t = torch()
    from blockwise_scaled_fp8_quant_amd.rotary import Rotary, rotary, rotary_frequencies
    x = t.randn((33, 4, 32), device="cuda")
    want = rotary(x, rotary_frequencies(32)[0].cuda())
    module = Rotary(32)
    with t.inference_mode():
        assert t.equal(module(x), want)
    leaf = x.clone().requires_grad_(True)
    y = module(leaf)
    assert t.equal(y, want)
    dy = t.randn_like(x)
    y.backward(dy)
    # the turn back, with the same frequencies: bit for bit the inverse call
    assert t.equal(leaf.grad, P.puro_rotary(dy, rotary_frequencies(32)[0].cuda(), inverse=True))


def test_first_call_under_a_capture_is_refused(P):
    t = torch()
    from blockwise_scaled_fp8_quant_amd.rotary import Rotary
    x = t.randn((7, 2, 16), device="cuda")
    cold, warm, here = Rotary(16), Rotary(16), Rotary(16, device="cuda")
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        want = warm(x)
    t.cuda.current_stream().wait_stream(side)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="being captured"):
            cold(x)
        y, z = warm(x), here(x)
    for k in range(3):
        x.add_(1.0)
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(y, warm(x)) and t.equal(z, here(x)), k
    assert want.shape == y.shape and t.equal(cold(x), y)
