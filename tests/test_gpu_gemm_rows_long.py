"""GPU tests of long products of any number of rows: which rows the blockwise GEMM may take, and what the others keep."""
import pytest

from gpu_util import say, torch
from test_gpu_gemm_rows import check, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


@pytest.mark.parametrize("M", [32768 + 3, 32768 + 130])
def test_weights_that_32_bit_offsets_do_not_reach(P, M):
    """2^33 multiplications and more with weight rows 2^24 apart and row scales that are not a multiple of four: the
    blockwise GEMM's kernel for such weights would read the scales of four rows at once, off 16 bytes."""
    t = torch()
    N, K = 128, 2048
    A, sA, B, sB = operands(M, N, K, M)
    wide = t.empty(N << 24, dtype=t.uint8, device="cuda").as_strided((N, K), (1 << 24, 1))
    wide.copy_(B)
    say(f"[rows, far weights] {M}x{N}x{K}")
    check(P, A, sA, B, sB, P.puro_gemm_rows(A, sA, wide, sB), t.bfloat16, "far weights")


def test_row_scales_on_four_bytes(P):
    """Where the four-wave kernel reaches, row scales may start at any element."""
    t = torch()
    A, sA, B, sB = operands(2048, 2048, 2048, 5)
    off = t.empty(sA.numel() + 1, device="cuda")[1:].view(sA.shape)
    off.copy_(sA)
    assert off.data_ptr() % 16 == 4 and t.equal(P.puro_gemm_rows(A, off, B, sB), P.puro_fp8_gemm(P.FWD, A, sA, B, sB))


@pytest.mark.parametrize("M", [128, 130, 200, 255])
def test_half_a_row_of_tiles_needs_twice_the_product(P, M):
    """128 to 255 rows: the blockwise GEMM takes 128 of them from 2^34 multiplications; below, every row keeps the row
    kernel's bound."""
    t = torch()
    A, sA, B, sB = operands(M, 8192, 8192, M)
    say(f"[rows, half a tile row] {M}x8192x8192")
    check(P, A, sA, B, sB, P.puro_gemm_rows(A, sA, B, sB), t.bfloat16, "below")
    A, sA, B, sB = operands(M, 16384, 8192, M)
    C = P.puro_gemm_rows(A, sA, B, sB)
    assert t.equal(C[:128], P.puro_fp8_gemm(P.FWD, A[:128], sA[:, :128].contiguous(), B, sB))
    if M > 128:
        check(P, A[128:], sA[:, 128:].contiguous(), B, sB, C[128:], t.bfloat16, "rest")
