"""GPU tests of the norm of rows that have no columns: their statistics, 0 / 0, are written."""
import pytest

from gpu_util import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


def test_statistics_of_no_columns(P):
    t = torch()
    x, w = t.empty((256, 0), device="cuda"), t.empty(0, device="cuda")
    stats = lambda: (t.full((256,), 7.0, device="cuda"), t.full((256,), 7.0, device="cuda"))
    for kind in (0, 1):
        m, r = stats()
        given = dict(mean=None if kind else m, rstd=r)
        for call in (lambda: P.puro_layer_norm(x, w, kind=kind, **given), lambda: P.puro_layer_norm_quant_dual(x, w, kind=kind, **given),
                     lambda: P.puro_layer_norm_quant(x, w, kind=kind, **given)):
            m.fill_(7)
            r.fill_(7)
            call()
            assert r.isnan().all() and (kind or m.isnan().all())
        for made in (P.puro_layer_norm(x, w, kind=kind)[1:], P.puro_layer_norm_quant_dual(x, w, kind=kind)[4:]):
            assert made[1].isnan().all() and (made[0] is None if kind else made[0].isnan().all())
