"""Which entry points Fp8Linear calls without gradients (no GPU: the calls are recorded), and that they give the
differentiable call's result."""
import pytest

from gpu_util import torch


def test_no_codes_for_a_backward_pass(monkeypatch):
    t = torch()
    from blockwise_scaled_fp8_quant_amd import linear
    calls = []

    def fake(name, result):
        def call(*a, **k):
            calls.append((name, k))
            return result(*a)
        monkeypatch.setattr(linear, name, call)
    fake("puro_fp8_quant_act_1x128", lambda x: (x, None))
    fake("puro_fp8_quant_act_dual", lambda x: (x, None, None, None))
    fake("puro_fp8_quant_w_128x128", lambda w: (w, None, None, None))
    fake("puro_fp8_gemm", lambda mode, a, sa, b, sb, **k: t.zeros(a.shape[0], b.shape[0]))
    fake("puro_gemm_rows", lambda a, sa, b, sb: t.zeros(a.shape[0], b.shape[0]))
    lin = linear.Fp8Linear(256, 384)
    with t.no_grad():
        for rows, product in ((128, "puro_fp8_gemm"), (256, "puro_fp8_gemm"), (0, "puro_fp8_gemm"), (1, "puro_gemm_rows"),
                              (129, "puro_gemm_rows")):
            calls.clear()
            assert lin(t.zeros(rows, 256, dtype=t.bfloat16)).shape == (rows, 384)
            assert [c[0] for c in calls] == ["puro_fp8_quant_act_1x128", "puro_fp8_quant_w_128x128", product]
            assert calls[1][1] == {"transposed": False}
        for bad, error in ((t.zeros(128, 128, dtype=t.bfloat16), ValueError), (t.zeros(128, 256), TypeError)):
            with pytest.raises(error):
                lin(bad)


@pytest.mark.gpu
def test_the_differentiable_calls_result():
    t = torch()
    from blockwise_scaled_fp8_quant_amd.linear import Fp8Linear
    for rows, din, dout in ((128, 256, 384), (1024, 512, 640), (4096, 2048, 2048)):
        lin = Fp8Linear(din, dout, device="cuda")
        x = t.randn((2, rows // 2, din), device="cuda").bfloat16()
        want = lin(x).detach()
        with t.no_grad():
            assert t.equal(lin(x), want)
