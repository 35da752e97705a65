"""GPU tests of the operators together, as a model uses them: norm + FP8 linear forward and backward, the serving
path for ragged rows, and the clipping of the gradients that come out."""
import pytest

from gpu_util import say, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def layer(P, kind, din=256, dout=384, seed=0):
    t = torch()
    from blockwise_scaled_fp8_quant_amd.norm import Fp8NormLinear
    t.manual_seed(seed)
    m = Fp8NormLinear(din, dout, kind=kind, device="cuda")
    with t.no_grad():
        for p in m.norm.parameters():
            p.add_(0.1 * t.randn_like(p))
    return m


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("xdtype", ["bfloat16", "float32"])
def test_training_step_is_the_chain_of_its_operators(P, kind, xdtype):
    """Outputs and gradients equal, bit for bit, the entry points called one after the other."""
    t = torch()
    m = layer(P, kind)
    m.enable_main_grad()
    x = t.randn((2, 128, 256), device="cuda").to(getattr(t, xdtype)).requires_grad_(True)
    dy = (t.randn((2, 128, 384), device="cuda") * 1e-2).bfloat16()
    y = m(x)
    y.backward(dy)
    n, w = m.norm, m.linear.weight
    x2, dy2 = x.detach().view(256, 256), dy.view(256, 384)
    q, s, qT, sT, mean, rstd = P.puro_layer_norm_quant_dual(x2, n.weight.detach(), None if kind else n.bias.detach(), eps=n.eps,
                                                            kind=kind)
    wq, ws, wqT, wsT = P.puro_fp8_quant_w_128x128(w.detach())
    assert t.equal(y.view(256, 384), P.puro_fp8_gemm(P.FWD, q, s, wq, ws))
    gq, gs, gqT, gsT = P.puro_fp8_quant_act_dual(dy2)
    dn = P.puro_fp8_gemm(P.DGRAD, gq, gs, wqT, wsT, out_dtype=P.OUT_BF16 if xdtype == "bfloat16" else P.OUT_FP32)
    dx, dw, db = P.puro_layer_norm_backward(dn, x2, n.weight.detach(), mean, rstd, kind=kind, with_bias=kind == 0)
    assert t.equal(x.grad.view(256, 256), dx)
    assert t.equal(n.weight.main_grad, dw) and n.weight.grad is None
    if kind == 0:
        assert t.equal(n.bias.main_grad, db)
    assert t.equal(w.main_grad, P.puro_fp8_gemm(P.WGRAD, gqT, gsT, qT, sT, out_dtype=P.OUT_FP32))
    # a second micro-batch adds one fp32 sum per element
    kept = n.weight.main_grad.clone()
    x.grad = None
    m(x).backward(dy)
    assert t.equal(n.weight.main_grad, kept + dw)


@pytest.mark.parametrize("kind", [0, 1])
def test_close_to_the_unquantized_layer(P, kind):
    """E4M3 keeps three mantissa bits: products of two quantized values are about 5% RMS off, 8% is the bound."""
    t = torch()
    m = layer(P, kind, 512, 640)
    x = t.randn((256, 512), device="cuda").requires_grad_(True)
    dy = t.randn((256, 640), device="cuda").bfloat16()
    y = m(x)
    y.backward(dy)
    xf = x.detach().double().cpu().requires_grad_(True)
    g = m.norm.weight.detach().double().cpu().requires_grad_(True)
    w = m.linear.weight.detach().double().cpu().requires_grad_(True)
    d = xf - xf.mean(1, keepdim=True) if kind == 0 else xf
    h = d * (d.square().mean(1, keepdim=True) + m.norm.eps).rsqrt() * g
    if kind == 0:
        h = h + m.norm.bias.detach().double().cpu()
    ref = h @ w.t()
    ref.backward(dy.double().cpu())
    rel = lambda a, b: float((a.detach().double().cpu() - b).norm() / b.norm())
    errs = [rel(y, ref.detach()), rel(x.grad, xf.grad), rel(m.norm.weight.grad, g.grad), rel(m.linear.weight.grad, w.grad)]
    say(f"    kind {kind}: Y, dX, dg, dW off by {errs}")
    assert max(errs) < 0.08


def test_serving_any_number_of_rows(P):
    t = torch()
    from blockwise_scaled_fp8_quant_amd.linear import Fp8Linear
    m = layer(P, 1)
    lin = Fp8Linear(256, 384, device="cuda")
    with t.no_grad():
        codes, lcodes = m.quantize_weight(), lin.quantize_weight()
        whole = t.randn((256, 256), device="cuda").bfloat16()
        for rows in (1, 3, 100, 129, 256):
            x = whole[:rows].view(1, rows, 256)
            y = m(x, codes)
            q, s = P.puro_layer_norm_quant(x[0], m.norm.weight, eps=m.norm.eps, kind=1)
            assert y.shape == (1, rows, 384) and t.equal(y[0], P.puro_gemm_rows(q, s, *codes))
            z = lin(x, lcodes)
            assert t.equal(z[0], P.puro_gemm_rows(*P.puro_fp8_quant_act_1x128(x[0]), *lcodes))
            assert t.equal(m(x), y)
            if rows % 128:
                assert t.equal(lin(x), z)
        assert m(whole[:0], codes).shape == (0, 384) and m(whole[:0]).shape == (0, 384)
    with pytest.raises(ValueError):
        lin(whole, lcodes)                                       # codes are not differentiable
    with pytest.raises(ValueError):
        m(whole, codes)
    for wide in (whole.view(128, 512), whole[:, :128].contiguous()):
        with pytest.raises(ValueError):
            m(wide)                                              # as many elements do not make it the width
        with t.no_grad(), pytest.raises(ValueError):
            m(wide, codes)
    with pytest.raises(P.PuroError):
        m(whole[:100])                                           # a ragged training batch


def test_norm_module_gradients(P):
    """The module's gradients against PyTorch's in 64 bits; fp32 sums and at most one rounding to bf16 (2^-8)."""
    t = torch()
    from blockwise_scaled_fp8_quant_amd.norm import Norm, layer_norm, rms_norm
    for kind in (0, 1):
        n = Norm(200, kind, dtype=t.float32, device="cuda")
        x = t.randn((3, 7, 200), device="cuda", requires_grad=True)
        dy = t.randn((3, 7, 200), device="cuda")
        y = n(x)
        y.backward(dy)
        xf = x.detach().double().requires_grad_(True)
        wf = n.weight.detach().double().requires_grad_(True)
        d = xf - xf.mean(-1, keepdim=True) if kind == 0 else xf
        ref = d * (d.square().mean(-1, keepdim=True) + n.eps).rsqrt() * wf
        ref.backward(dy.double())
        for a, b in ((y, ref), (x.grad, xf.grad), (n.weight.grad, wf.grad)):
            assert (a.detach().double() - b.detach()).abs().max() <= 200 * 2.0 ** -24 * b.detach().abs().max()
    x = t.randn((5, 64), device="cuda")
    w = t.ones(64, device="cuda")
    assert t.equal(layer_norm(x, w), P.puro_layer_norm(x, w)[0])
    assert t.equal(rms_norm(x, w), P.puro_layer_norm(x, w, eps=1e-6, kind=P.RMS_NORM)[0])


def test_broadcast_gradients_and_changed_weights(P):
    """A gradient broadcast over rows (of a sum over them) is taken; a weight changed between the passes is refused;
    so is a second derivative."""
    t = torch()
    from blockwise_scaled_fp8_quant_amd.norm import Norm
    n = Norm(256, 0, device="cuda")
    x = t.randn((128, 256), device="cuda").bfloat16().requires_grad_(True)
    g = t.randn(256, device="cuda").bfloat16()
    n(x).sum(0).backward(g)
    dx, n.weight.grad, n.bias.grad, x.grad = x.grad, None, None, None
    n(x).backward(g.expand(128, 256).contiguous())
    assert t.equal(dx, x.grad)
    m = layer(P, 1)
    x = t.randn((128, 256), device="cuda").bfloat16().requires_grad_(True)
    m(x).sum(0).backward(t.ones(384, device="cuda").bfloat16())
    assert x.grad.isfinite().all()
    for mod, param in ((n, n.weight), (m, m.norm.weight)):
        y = mod(x)
        with t.no_grad():
            param.mul_(2)
        with pytest.raises(RuntimeError):
            y.backward(t.ones_like(y))
    y = n(x)
    (first,) = t.autograd.grad(y.float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        first.float().sum().backward()


def test_frozen_parameters_get_nothing(P):
    t = torch()
    m = layer(P, 0)
    m.enable_main_grad()
    m.norm.weight.requires_grad_(False)
    x = t.randn((128, 256), device="cuda").bfloat16().requires_grad_(True)
    m(x).backward(t.ones((128, 384), device="cuda").bfloat16())
    assert (m.norm.weight.main_grad == 0).all() and (m.norm.bias.main_grad != 0).any() and x.grad is not None
    m.norm.bias.requires_grad_(False)
    kept = m.norm.bias.main_grad.clone()
    m(x).backward(t.ones((128, 384), device="cuda").bfloat16())
    assert t.equal(m.norm.bias.main_grad, kept)


def test_step_with_clipping(P):
    """Forward, backward and clipping of two stacked layers: afterwards the global norm is the bound."""
    t = torch()
    from blockwise_scaled_fp8_quant_amd.clip import clip_grad_norm_, gradients
    a, b = layer(P, 0, 256, 384, 1), layer(P, 1, 384, 256, 2)
    for m in (a, b):
        m.enable_main_grad()
    x = t.randn((256, 256), device="cuda").bfloat16()
    b(a(x)).backward((t.randn((256, 256), device="cuda")).bfloat16())
    params = list(a.parameters()) + list(b.parameters())
    grads = gradients(params)
    assert len(grads) == 5 and all(g.dtype == t.float32 for g in grads)
    before = [g.clone() for g in grads]
    norm = clip_grad_norm_(params, 0.25)
    ref = sum(float(g.double().square().sum()) for g in before) ** 0.5
    assert abs(float(norm) / ref - 1) <= 2.0 ** -23 and ref > 0.25
    for g, o in zip(grads, before):
        assert (g.double() - o.double() * (0.25 / (ref + 1e-6))).abs().max() <= 6 * 2.0 ** -24 * g.abs().max().double()
    assert abs(float(P.puro_grad_norm(grads)) - 0.25) < 1e-6


@pytest.mark.parametrize("kind", [0, 1])
def test_step_in_a_graph(P, kind):
    """Forward, backward and clipping captured together; every replay against an eager step on other inputs."""
    import copy
    t = torch()
    from blockwise_scaled_fp8_quant_amd.clip import clip_grad_norm_
    m = layer(P, kind)
    m.enable_main_grad()
    e = copy.deepcopy(m)
    e.enable_main_grad()
    xin = t.randn((128, 256), device="cuda").bfloat16().requires_grad_(True)
    dyin = t.randn((128, 384), device="cuda").bfloat16()

    def step(mod, x, dy):
        for p in mod.parameters():
            p.main_grad.zero_()
        y = mod(x)
        y.backward(dy)
        return y.detach(), clip_grad_norm_(mod.parameters(), 0.5)

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step(m, xin, dyin)
    t.cuda.current_stream().wait_stream(side)
    xin.grad = None
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        y, norm = step(m, xin, dyin)
    x0, dy0 = xin.detach().clone(), dyin.clone()
    for k in range(3):
        with t.no_grad():
            xin.copy_(x0 * (k + 1) - k)
            dyin.copy_(dy0 / (k + 1))
        graph.replay()
        t.cuda.synchronize()
        x = xin.detach().clone().requires_grad_(True)
        ey, enorm = step(e, x, dyin)
        assert t.equal(y, ey) and t.equal(norm, enorm) and t.equal(xin.grad, x.grad), k
        for a, b in zip(m.parameters(), e.parameters()):
            assert a.main_grad.any() and t.equal(a.main_grad, b.main_grad), k


def test_capture_over_a_living_graph_is_refused(P):
    t = torch()
    from blockwise_scaled_fp8_quant_amd.norm import Norm
    m, n = layer(P, 1), Norm(256, 0, device="cuda")
    x = t.randn((128, 256), device="cuda").bfloat16()
    living = [m(x), n(x)]
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        out = x * 2
        for mod in (m, n):
            with pytest.raises(RuntimeError, match="captured"):
                mod(x)
        with t.no_grad():
            y = n(x)                                             # without gradients there is nothing to join
    graph.replay()
    t.cuda.synchronize()
    assert t.equal(out, x * 2) and t.equal(y, n(x).detach())
    for z in living:
        z.backward(t.ones_like(z))                               # the eager graphs are as they were
    assert n.weight.grad.isfinite().all() and m.linear.weight.grad.isfinite().all()
