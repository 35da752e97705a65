"""GPU tests of the blockwise GEMM on operands that end with their last code or scale: a second launch over the last 128
rows, and rows that are further apart than their codes."""
import pytest

from gpu_util import say, torch
from test_gpu_gemm_rows import operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


@pytest.mark.parametrize("M,N,K", [(8320, 2048, 16384), (384, 256, 1024), (256, 384, 2048)])
def test_operands_that_end_with_their_last_row(P, M, N, K):
    """Rows 64 codes further apart than they are long, the last one ending its allocation: as contiguous ones, bit for bit."""
    t = torch()
    A, sA, B, sB = operands(M, N, K, M)

    def last_row_ends(q):
        ld = K + 64
        buf = t.empty((q.shape[0] - 1) * ld + K, dtype=t.uint8, device="cuda")
        v = buf.as_strided(q.shape, (ld, 1))
        v.copy_(q)
        return v
    a, b = last_row_ends(A), last_row_ends(B)
    say(f"[reach] {M}x{N}x{K}")
    for dtype in (P.OUT_BF16, P.OUT_FP32):
        want = P.puro_fp8_gemm(P.FWD, A, sA, B, sB, out_dtype=dtype)
        assert t.equal(P.puro_fp8_gemm(P.FWD, a, sA, b, sB, out_dtype=dtype), want)
        assert t.equal(P.puro_fp8_gemm(P.DGRAD, a, sA, b, sB, out_dtype=dtype), want)
        # the last 128 rows on their own: the sums may be split otherwise, so up to a normalized error of 1e-3
        few = P.puro_fp8_gemm(P.FWD, A[-128:], sA[:, -128:].contiguous(), B, sB, out_dtype=dtype).float()
        norm = lambda q, s: (q.view(t.float8_e4m3fn).float() * s).norm(dim=1)
        den = norm(A[-128:], sA[:, -128:].t().repeat_interleave(128, 1))[:, None] * \
            norm(B, sB.repeat_interleave(128, 0).repeat_interleave(128, 1))[None, :]
        assert ((few - want[-128:].float()).abs() <= 1e-3 * den).all()
