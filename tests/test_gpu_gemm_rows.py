"""GPU tests of the few-row FP8 product, against the sum of the decoded products in 64 bits.

Tolerance, with u = 2^-24: products of two E4M3 values are exact in fp32; a slice's sum of 128 has under 128
roundings, its scaling two, the sum over K / 128 slices one each, joining 8 waves 8 (and as many for the parts of a split):
(160 + K / 128) u sum|a b| s, then half a step of the output type."""
import pytest

from gpu_util import say, torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def operands(M, N, K, seed, lda=0, ldb=0):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    def codes(r, c, ld):
        # every finite code byte
        q = t.randint(0, 254, (r, max(c, ld)), generator=g, device="cuda")
        q = (q + (q >= 127)).to(t.uint8)
        return q[:, :c]
    A, B = codes(M, K, lda), codes(N, K, ldb)
    sA = t.exp2(t.rand((K // 128, M), generator=g, device="cuda") * 8 - 12)
    sB = t.exp2(t.rand((N // 128, K // 128), generator=g, device="cuda") * 8 - 12)
    return A, sA, B, sB


def reference(A, sA, B, sB):
    t = torch()
    a = A.contiguous().view(t.float8_e4m3fn).double() * sA.double().t().repeat_interleave(128, 1)
    b = B.contiguous().view(t.float8_e4m3fn).double() * sB.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    return a @ b.t(), a.abs() @ b.abs().t()


def check(P, A, sA, B, sB, C, dtype, what):
    t = torch()
    ref, size = reference(A, sA, B, sB)
    bound = (160 + A.shape[1] / 128) * U * size
    if dtype == t.bfloat16:
        bound = bound * (1 + 2.0 ** -7) + ref.abs() * (t.finfo(dtype).eps / 2)
    d = (C.double() - ref).abs()
    assert (d <= bound).all(), (what, float((d / bound.clamp_min(1e-300)).max()))
    return float((C.double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("N,K", [(128, 128), (256, 384), (640, 1152), (2048, 2048), (128, 6144)])
def test_every_row_count(P, N, K):
    t = torch()
    rows = list(range(1, 36)) + [47, 48, 49, 63, 64, 65, 96, 127, 128, 129, 200, 256, 257] if N <= 256 else [1, 2, 15, 16, 17, 33, 70, 131]
    for M in rows:
        A, sA, B, sB = operands(M, N, K, M + N + K)
        say(f"[rows] M,N,K={M},{N},{K}")
        e32 = check(P, A, sA, B, sB, P.puro_gemm_rows(A, sA, B, sB, out_dtype=P.OUT_FP32), t.float32, (M, N, K))
        check(P, A, sA, B, sB, P.puro_gemm_rows(A, sA, B, sB), t.bfloat16, (M, N, K))
    say(f"    fp32 relative error {e32:.2e}")


@pytest.mark.parametrize("M,N,K", [(1061, 4096, 2048), (1024, 512, 16384), (1026, 512, 16512)])
def test_long_products(P, M, N, K):
    """Leading rows of a long bf16 product are the blockwise GEMM's, bit for bit, with a contraction split and
    without; the rest, and an fp32 output throughout, keep the bound above."""
    t = torch()
    A, sA, B, sB = operands(M, N, K, 2)
    lead = M - M % 128
    C = P.puro_gemm_rows(A, sA, B, sB)
    want = P.puro_fp8_gemm(P.FWD, A[:lead], sA[:, :lead].contiguous(), B, sB)
    assert t.equal(C[:lead], want)
    if lead < M:
        check(P, A[lead:], sA[:, lead:].contiguous(), B, sB, C[lead:], t.bfloat16, "rest")
    check(P, A, sA, B, sB, P.puro_gemm_rows(A, sA, B, sB, out_dtype=P.OUT_FP32), t.float32, "fp32")


def test_strides_and_gaps(P):
    t = torch()
    for M, N, K in ((5, 256, 256), (40, 384, 512), (130, 128, 256)):
        A, sA, B, sB = operands(M, N, K, M, lda=K + 48, ldb=K + 16)
        C = t.full((M + 2, N + 24), 5.0, dtype=t.bfloat16, device="cuda")
        P.puro_gemm_rows(A, sA, B, sB, C=C[1:M + 1, 8:N + 8])
        check(P, A, sA, B, sB, C[1:M + 1, 8:N + 8], t.bfloat16, "strided")
        C[1:M + 1, 8:N + 8] = 5.0
        assert (C == 5).all()


def test_single_row_and_column_views(P):
    """Dimensions of one element may carry any stride: one row's scales are a column however they were made."""
    t = torch()
    A, sA, B, sB = operands(1, 128, 512, 4)
    want = P.puro_gemm_rows(A, sA, B, sB)
    odd = sA.t().contiguous().t()
    assert odd.shape == sA.shape and t.equal(P.puro_gemm_rows(A.expand(1, 512), odd, B, sB), want)
    wide = t.zeros((3, 512), dtype=t.uint8, device="cuda")
    wide[1] = A[0]
    assert t.equal(P.puro_gemm_rows(wide[1:2], sA, B, sB), want)


def test_exact_integers(P):
    """Small integers with power-of-two scales: every partial sum is exact, so the result is."""
    t = torch()
    for M, N, K in ((1, 128, 256), (19, 256, 1024), (100, 128, 640)):
        a = t.randint(-3, 4, (M, K), device="cuda").float()
        b = t.randint(-3, 4, (N, K), device="cuda").float()
        A, B = a.to(t.float8_e4m3fn).view(t.uint8), b.to(t.float8_e4m3fn).view(t.uint8)
        sA, sB = t.full((K // 128, M), 0.5, device="cuda"), t.full((N // 128, K // 128), 4.0, device="cuda")
        C = P.puro_gemm_rows(A, sA, B, sB, out_dtype=P.OUT_FP32)
        assert t.equal(C.double(), 2 * (a.double() @ b.double().t()))


def test_agrees_with_the_quantizers_and_the_blockwise_product(P):
    """M = 256 rows through both products: the same sums up to both tolerances (1e-4 of the norms for the FP8 one)."""
    t = torch()
    x, w = t.randn(256, 1024, device="cuda").bfloat16(), (t.randn(512, 1024, device="cuda") * 0.02).bfloat16()
    q, s = P.puro_fp8_quant_act_1x128(x)
    wq, ws, _, _ = P.puro_fp8_quant_w_128x128(w)
    a = P.puro_fp8_gemm(P.FWD, q, s, wq, ws, out_dtype=P.OUT_FP32)
    b = P.puro_gemm_rows(q, s, wq, ws, out_dtype=P.OUT_FP32)
    ra, _ = reference(q, s, wq, ws)
    den = x.float().norm(dim=1)[:, None] * w.float().norm(dim=1)[None, :]
    assert ((a - b).abs() <= 2e-4 * den).all()
    # rows are independent of how many there are
    few = P.puro_gemm_rows(q[:5].contiguous(), s[:, :5].contiguous(), wq, ws, out_dtype=P.OUT_FP32)
    assert ((few - b[:5]).abs() <= 1e-5 * den[:5]).all()


def test_nan_codes_stay_in_their_row_and_column(P):
    t = torch()
    A, sA, B, sB = operands(20, 256, 256, 1)
    clean = P.puro_gemm_rows(A, sA, B, sB, out_dtype=P.OUT_FP32)
    A[3, 100] = 0x7F
    B[200, 7] = 0xFF
    C = P.puro_gemm_rows(A, sA, B, sB, out_dtype=P.OUT_FP32)
    bad = t.zeros_like(C, dtype=t.bool)
    bad[3] = bad[:, 200] = True
    assert C[bad].isnan().all() and t.equal(C[~bad], clean[~bad])


def test_empty(P):
    t = torch()
    u8 = lambda *s: t.empty(s, dtype=t.uint8, device="cuda")
    f = lambda *s: t.empty(s, device="cuda")
    assert P.puro_gemm_rows(u8(0, 128), f(1, 0), u8(128, 128), f(1, 1)).shape == (0, 128)
    C = t.ones((3, 128), device="cuda", dtype=t.bfloat16)
    P.puro_gemm_rows(u8(3, 0), f(0, 3), u8(128, 0), f(1, 0), C=C)
    assert (C == 0).all()


def test_graph_and_stream(P):
    t = torch()
    for M, N, K in ((1, 2048, 2048), (45, 512, 6144)):
        A, sA, B, sB = operands(M, N, K, 3)
        want = P.puro_gemm_rows(A, sA, B, sB)
        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        got = P.puro_gemm_rows(A, sA, B, sB, stream=side)
        t.cuda.synchronize()
        assert t.equal(want, got)
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            out = P.puro_gemm_rows(A, sA, B, sB)
        for k in range(3):
            sA.mul_(1.5)
            graph.replay()
            t.cuda.synchronize()
            assert t.equal(out, P.puro_gemm_rows(A, sA, B, sB)), k


def test_refusals(P):
    t = torch()
    A, sA, B, sB = operands(3, 256, 256, 1)
    with pytest.raises(ValueError):
        P.puro_gemm_rows(A, sA.t().contiguous(), B, sB)
    with pytest.raises(ValueError):
        P.puro_gemm_rows(A, sA, B[:, :128], sB)
    with pytest.raises(TypeError):
        P.puro_gemm_rows(A.view(t.int8), sA, B, sB)
    with pytest.raises(ValueError):
        P.puro_gemm_rows(A, sA, B, sB, out_dtype=4)
    with pytest.raises(P.PuroError):
        P.puro_gemm_rows(A[:, :100], sA[:0], B[:, :100], sB[:, :0])
    with pytest.raises(P.PuroError):
        P.puro_gemm_rows(A, sA, B[:200], sB[:1])


def test_weights_past_32_bit_offsets(P):
    """Weight rows whose codes lie more than 2^31 bytes apart, and an output whose rows do."""
    t = torch()
    ld = (1 << 26) + 16
    big = t.zeros(128 * ld, dtype=t.uint8, device="cuda")
    A, sA, B, sB = operands(2, 128, 256, 8)
    wide = big.as_strided((128, 256), (ld, 1))
    wide.copy_(B)
    assert t.equal(P.puro_gemm_rows(A, sA, wide, sB), P.puro_gemm_rows(A, sA, B, sB))
    out = big[: 128 * ld // 32 * 32].view(t.bfloat16).as_strided((2, 128), ((1 << 31) + 64, 1), 0)
    P.puro_gemm_rows(A, sA, B, sB, C=out)
    assert t.equal(out, P.puro_gemm_rows(A, sA, B, sB))


def test_more_fp32_rows_than_a_launch_holds(P):
    """The rows on both sides of the limit and the last ones, as by themselves (one slice: any split sums alike)."""
    t = torch()
    M = 65535 * 64 + 3
    A, sA, B, sB = operands(64, 128, 128, 9)
    reps = M // 64 + 1
    A, sA = A.repeat(reps, 1)[:M], sA.repeat(1, reps)[:, :M].contiguous()
    say(f"[rows, large] {M}x128x128 fp32")
    C = P.puro_gemm_rows(A, sA, B, sB, out_dtype=P.OUT_FP32)
    ref = P.puro_gemm_rows(A[:64], sA[:, :64].contiguous(), B, sB, out_dtype=P.OUT_FP32)
    assert ref.any() and t.equal(C[:M // 64 * 64].view(-1, 64, 128), ref.expand(M // 64, 64, 128))
    assert t.equal(C[-3:], ref[:3])


# one shape for each tile and split over waves of the kernel, most with columns and rows left over
@pytest.mark.parametrize("M,N", [(1, 128), (1, 4224), (1, 8320), (1, 16512), (3, 12416), (5, 24704), (34, 1408), (19, 6272),
                                 (19, 8320), (19, 16512), (19, 12416), (19, 24704), (67, 1664), (34, 6272), (34, 8320),
                                 (34, 16512), (34, 12416), (34, 24704), (145, 2560), (49, 8320), (49, 16512), (49, 12416),
                                 (49, 24704), (300, 12416)])
def test_every_tile(P, M, N):
    """A contraction that leaves some waves a slice less, and some none."""
    t = torch()
    for K in (384, 1152, 2432):
        A, sA, B, sB = operands(M, N, K, M + N)
        say(f"[rows] M,N,K={M},{N},{K}")
        check(P, A, sA, B, sB, P.puro_gemm_rows(A, sA, B, sB, out_dtype=P.OUT_FP32), t.float32, (M, N, K))
        check(P, A, sA, B, sB, P.puro_gemm_rows(A, sA, B, sB), t.bfloat16, (M, N, K))
