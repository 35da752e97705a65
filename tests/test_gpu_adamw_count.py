"""GPU tests of the count of steps that a capturable AdamW keeps on the GPU: a refused step is none."""
import pytest

from gpu_util import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def P():
    import blockwise_scaled_fp8_quant_amd as P
    assert torch().cuda.is_available(), "GPU test run without a GPU"
    return P


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [True, False])
def test_refused_steps_are_not_counted(P, bits, capturable):
    """After steps that are refused for a rate, betas, a bound or a type, the next one gives the bits of an optimizer that never
    saw them."""
    t = torch()
    from blockwise_scaled_fp8_quant_amd.adamw import AdamW
    start, grads = t.randn(300, device="cuda"), [t.randn(300, device="cuda") * 1e-2 for _ in range(3)]

    def make():
        p = t.nn.Parameter(start.clone())
        return p, AdamW([p], lr=1e-2, state_bits=bits, seed=3, capturable=capturable)
    (p, opt), (q, other) = make(), make()
    for k, g in enumerate(grads):
        p.grad = q.grad = g
        group = opt.param_groups[0]
        for name, bad, error in (("lr", float("nan"), P.PuroError), ("betas", (1.0, 0.9), P.PuroError), ("lr", "much", TypeError),
                                 ("lr", t.ones(1, device="cuda").double(), TypeError)):
            kept, group[name] = group[name], bad
            with pytest.raises(error):
                opt.step()
            group[name] = kept
        with pytest.raises(P.PuroError):
            opt.step(max_norm=-1.0)
        assert int(opt.state[p]["step"]) == k
        opt.step()
        other.step()
        assert int(opt.state[p]["step"]) == k + 1 and t.equal(p, q)
        for name in ("exp_avg", "exp_avg_sq"):
            assert t.equal(opt.state[p][name], other.state[q][name])


def test_a_step_refused_under_a_capture_is_not_counted_by_replays(P):
    t = torch()
    from blockwise_scaled_fp8_quant_amd.adamw import AdamW
    p, q = (t.nn.Parameter(t.ones(300, device="cuda")) for _ in range(2))
    opt, other = AdamW([p], lr=1e-2, capturable=True), AdamW([q], lr=1e-2, capturable=True)
    p.grad, q.grad = (t.full((300,), 0.5, device="cuda") for _ in range(2))
    opt.step()
    other.step()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        opt.param_groups[0]["lr"] = float("nan")
        with pytest.raises(P.PuroError):
            opt.step()
        opt.param_groups[0]["lr"] = 1e-2
        opt.step()
    for k in range(3):
        graph.replay()
        other.step()
        t.cuda.synchronize()
        assert int(opt.state[p]["step"]) == int(other.state[q]["step"]) == k + 2 and t.equal(p, q)
