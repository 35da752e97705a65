"""The package without its native marshalling (not built, or not loadable): the entry points of puro_fp8.h load and
work, those of puro_ops.h say what is missing."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "blockwise_scaled_fp8_quant_amd"

PROGRAM = """
import torch
import blockwise_scaled_fp8_quant_amd as P
from blockwise_scaled_fp8_quant_amd.linear import Fp8Linear
from blockwise_scaled_fp8_quant_amd import norm, clip
assert P.puro_fp8_gemm_workspace_size(P.FWD, 128, 128, 128) >= 0 and P.puro_gemm_rows_workspace_size(1, 128, 128) == 0
x = torch.zeros(128, 128, dtype=torch.bfloat16)
for call, error in ((lambda: P.puro_fp8_quant_act_1x128(x), ValueError), (lambda: Fp8Linear(128, 128)(x), ValueError),
                    (lambda: P.puro_layer_norm(x, x[0]), ImportError), (lambda: P.puro_gemm_rows(x, x, x, x), ImportError),
                    (lambda: P.puro_clip_grad_norm([x], 1.0), ImportError), (lambda: norm.Norm(128)(x), ImportError)):
    try:
        call()
    except error as e:
        assert error is not ImportError or "_marshal.so" in str(e)
        continue
    raise SystemExit("not refused")
print("loaded")
"""


@pytest.mark.parametrize("built", ["missing", "broken"])
def test_package_loads(tmp_path, built):
    pkg = tmp_path / PKG
    pkg.mkdir()
    for name in os.listdir(os.path.join(ROOT, PKG)):
        if name.endswith(".py"):
            shutil.copy(os.path.join(ROOT, PKG, name), pkg / name)
    os.symlink(os.path.join(ROOT, PKG, "libpuro_fp8.so"), pkg / "libpuro_fp8.so")
    if built == "broken":
        (pkg / "_marshal.so").write_bytes(b"no library")
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "loaded", r.stderr[-2000:]
