"""GPU tests of the FP8 linear layer's step in a graph."""
import pytest

from gpu_util import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def test_capture_over_a_living_graph_is_refused(P):
    """An eager pass's living graph belongs to its stream: a captured pass over the same weight or input would end the
    process in the autograd engine, and is refused before it starts.  Without gradients there is nothing to join."""
    t = torch()
    from blockwise_scaled_fp8_quant_amd.linear import Fp8Linear, fp8_linear
    m = Fp8Linear(256, 384, device="cuda")
    x = t.randn((128, 256), device="cuda").bfloat16()
    xin = x.clone().requires_grad_(True)
    w = m.weight.detach().clone()
    living = [m(x), fp8_linear(xin, w)]
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        for call in (lambda: m(x), lambda: fp8_linear(x, m.weight), lambda: fp8_linear(xin, w)):
            with pytest.raises(RuntimeError, match="captured"):
                call()
        with t.no_grad():
            y = m(x)
    graph.replay()
    t.cuda.synchronize()
    assert t.equal(y, living[0].detach())
    for z in living:
        z.backward(t.ones_like(z))
    assert m.weight.grad.isfinite().all() and xin.grad.isfinite().all()


def test_capture_over_a_leaf_behind_a_view_is_refused(P):
    """What is given may be a view of such a leaf, or what an earlier operation made of one."""
    t = torch()
    from blockwise_scaled_fp8_quant_amd.linear import Fp8Linear
    from blockwise_scaled_fp8_quant_amd.norm import Norm, rms_norm
    m, n = Fp8Linear(256, 384, device="cuda"), Norm(256, 0, device="cuda")
    x = t.randn((2, 64, 256), device="cuda").bfloat16().requires_grad_(True)
    scale = t.ones(256, device="cuda").bfloat16().requires_grad_(True)
    fresh = t.randn((128, 256), device="cuda").bfloat16()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        m(fresh).backward(t.ones((128, 384), device="cuda").bfloat16())
    t.cuda.current_stream().wait_stream(side)
    m.weight.grad = None
    living = (x * 2, scale * 2)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        for call in (lambda: m(x.view(128, 256)), lambda: n((x + 1).flatten(0, 1)), lambda: rms_norm(fresh, scale.view(256)),
                     lambda: m((fresh * scale).contiguous())):
            with pytest.raises(RuntimeError, match="captured"):
                call()
        y = m(fresh)                              # nothing living reaches this one
        y.backward(t.ones_like(y))
    graph.replay()
    t.cuda.synchronize()
    assert m.weight.grad.isfinite().all() and len(living) == 2


def test_step_in_a_graph(P):
    """Forward and backward captured together after a pass whose graph is gone; every replay against an eager step."""
    import copy
    t = torch()
    from blockwise_scaled_fp8_quant_amd.linear import Fp8Linear
    m = Fp8Linear(256, 384, device="cuda")
    m.enable_main_grad()
    e = copy.deepcopy(m)
    e.enable_main_grad()
    xin = t.randn((128, 256), device="cuda").bfloat16().requires_grad_(True)
    dyin = t.randn((128, 384), device="cuda").bfloat16()

    def step(mod, x, dy):
        mod.weight.main_grad.zero_()
        y = mod(x)
        y.backward(dy)
        return y.detach()

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step(m, xin, dyin)
    t.cuda.current_stream().wait_stream(side)
    xin.grad = None
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        y = step(m, xin, dyin)
    x0, dy0 = xin.detach().clone(), dyin.clone()
    for k in range(3):
        with t.no_grad():
            xin.copy_(x0 * (k + 1) - k)
            dyin.copy_(dy0 / (k + 1))
        graph.replay()
        t.cuda.synchronize()
        x = xin.detach().clone().requires_grad_(True)
        assert t.equal(y, step(e, x, dyin)) and t.equal(xin.grad, x.grad), k
        assert m.weight.main_grad.any() and t.equal(m.weight.main_grad, e.weight.main_grad), k
