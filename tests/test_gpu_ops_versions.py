"""GPU tests that tensors a call writes have their version raised, so that autograd notices a saved one that changed."""
import pytest

from gpu_util import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def test_given_outputs_are_new_versions(P):
    t = torch()
    f = lambda *s: t.zeros(s, device="cuda")
    u8 = lambda *s: t.zeros(s, dtype=t.uint8, device="cuda")
    x, dy, w = t.randn((128, 256), device="cuda"), t.randn((128, 256), device="cuda"), f(256) + 1
    y, m, r = P.puro_layer_norm(x, w)
    q, s = P.puro_layer_norm_quant(x, w)
    wq, ws, _, _ = P.puro_fp8_quant_w_128x128(t.randn((384, 256), device="cuda").bfloat16())
    grads = [f(7) + 1, (f(9) + 1).bfloat16()]

    def raised(call, *given, kept=()):
        before = [g._version for g in given + kept]
        call(*given)
        after = [g._version for g in given + kept]
        assert all(b > a for a, b in zip(before[:len(given)], after)) and before[len(given):] == after[len(given):]
    raised(lambda y, m, r: P.puro_layer_norm(x, w, y=y, mean=m, rstd=r), f(128, 256), f(128), f(128), kept=(x, w))
    raised(lambda q, s, m, r: P.puro_layer_norm_quant(x, w, q=q, s=s, mean=m, rstd=r), u8(128, 256), f(2, 128), f(128), f(128))
    raised(lambda q, s, qT, sT, m, r: P.puro_layer_norm_quant_dual(x, w, q=q, s=s, qT=qT, sT=sT, mean=m, rstd=r),
           u8(128, 256), f(2, 128), u8(256, 128), f(1, 256), f(128), f(128))
    raised(lambda dx, dw, db: P.puro_layer_norm_backward(dy, x, w, m, r, dx=dx, dweight=dw, dbias=db, accumulate=True),
           f(128, 256), f(256), f(256), kept=(x, dy, w, m, r))
    raised(lambda C: P.puro_gemm_rows(q, s, wq, ws, C=C), f(128, 384).bfloat16(), kept=(q, s, wq, ws))
    raised(lambda n: P.puro_grad_norm(grads, norm=n), f(), kept=tuple(grads))
    raised(lambda *g: P.puro_clip_grad_norm(list(g), 0.5), *grads)
    raised(lambda *o: P.puro_clip_grad_norm(grads, 0.5, outs=list(o)), f(7), f(9).bfloat16(), kept=tuple(grads))
    raised(lambda *g: P.puro_scale_by_norm(list(g), 0.5, f() + 3), *grads)


def test_autograd_notices_what_was_overwritten(P):
    t = torch()
    x = t.randn((4, 64), device="cuda")
    p = t.randn((4, 64), device="cuda", requires_grad=True)
    z = p * x                                                  # keeps x
    P.puro_layer_norm(x, t.ones(64, device="cuda"), y=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()
    with t.inference_mode():                                   # tensors without a version
        v = t.randn((4, 64), device="cuda")
        y, _, _ = P.puro_layer_norm(v, t.ones(64, device="cuda"), y=t.zeros_like(v))
    P.puro_layer_norm(v, t.ones(64, device="cuda"), y=y)
    assert y.isfinite().all()
