"""The count of steps of an AdamW, on the host: a step that is refused (here for parameters that are not on the GPU) is none."""
import pytest
import torch

from blockwise_scaled_fp8_quant_amd.adamw import AdamW


@pytest.mark.parametrize("capturable", [True, False])
def test_refused_steps_are_not_counted(capturable, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)      # (asks a GPU otherwise)
    p = torch.nn.Parameter(torch.zeros(4))
    p.grad = torch.zeros(4)
    opt = AdamW([p], capturable=capturable)
    for _ in range(3):
        with pytest.raises(ValueError, match="GPU"):
            opt.step()
        assert int(opt.state[p]["step"]) == 0
