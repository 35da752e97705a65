"""The frequencies that a Rotary module keeps, on the host: whatever mode the first call on a device is made in, autograd may save
them later, and devices do not take each other's."""
import threading

import pytest
import torch

from blockwise_scaled_fp8_quant_amd.rotary import Rotary, rotary_frequencies


def test_frequencies_serve_autograd_after_inference_mode():
    with torch.inference_mode():
        module = Rotary(16)
        far = module.frequencies(torch.device("meta"))
    assert not module.frequencies(torch.device("cpu")).is_inference() and not far.is_inference()
    y = torch.ones(8, dtype=torch.float64, requires_grad=True) * module.frequencies(torch.device("cpu"))    # saves them
    y.sum().backward()
    with torch.inference_mode(), pytest.raises(ValueError):
        module(torch.zeros((2, 1, 16), device="meta"))              # (a call that is refused, but for its device)
    assert not module.frequencies(torch.device("meta")).is_inference()


def test_each_device_keeps_its_own():
    module = Rotary(16, base=500.0)
    cpu, meta = torch.device("cpu"), torch.device("meta")
    here = module.frequencies(cpu)
    assert torch.equal(here, rotary_frequencies(16, 500.0)[0])
    for _ in range(2):
        there = module.frequencies(meta)
        assert there.device == meta and module.frequencies(meta) is there and module.frequencies(cpu) is here
    assert module.half().frequencies(cpu).dtype == torch.float64 and not module.state_dict()


def test_threads_get_one_copy():
    module = Rotary(16)
    start, got = threading.Barrier(8), []

    def run():
        start.wait()
        got.append(module.frequencies(torch.device("meta")))
    threads = [threading.Thread(target=run) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 8 and all(f is got[0] for f in got)
