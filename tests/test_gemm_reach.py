"""What the four-wave kernels' buffer resources reach (CPU only): every code and scale of a tile's rows, and nothing
behind the matrix, for every launch of a plan.

A C++ program walks shapes whose plan has one or two launches, with rows as far apart as their codes and further, and
compares each tile's last reachable byte with the operand's last one: K codes of its last row, nothing of the gap behind
it; the last row's scale in the last slice."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "blockwise_scaled_fp8_quant_amd")

PROGRAM = r"""
#include <cstdio>
#include <cstdint>
#include "internal.hpp"
GEMM_REACH

int main() {
  long tiles = 0, second = 0;
  const int64_t Ms[] = {128, 256, 384, 1024, 8192, 8320, 8448, 11008, 12288, 16512};
  const int64_t Ns[] = {256, 2048, 8192};
  const int64_t Ks[] = {128, 2048, 16384, 32768};
  for (int64_t M : Ms)
    for (int64_t N : Ns)
      for (int64_t K : Ks)
        for (int64_t gap : {0, 16, 4096}) {
          const int64_t lda = K + gap, ldsa = M, nk = K / 128;
          const int64_t a_end = (M - 1) * lda + K, s_end = nk * M;     // bytes, scales
          puro::GemmPart parts[2];
          const int n = puro::gemm_parts(M, N, K, parts);
          for (int i = 0; i < n; ++i)
            for (int64_t m0 = 0; m0 < parts[i].rows; m0 += 256, ++tiles) {
              second += i;
              const int64_t row = parts[i].row0 + m0;
              const int left = (int)(parts[i].rows - m0);
              const int64_t last = row + (left < 256 ? left : 256) - 1;
              const int64_t a = row * lda + puro::tile_bytes(left, lda, (int)K);
              const int64_t s = row + puro::scale_bytes(left, ldsa, (int)K) / 4;
              if (a > a_end || a != last * lda + K) return std::printf("codes %ld %ld\n", (long)M, (long)m0), 1;
              if (s > s_end || s != (nk - 1) * ldsa + last + 1) return std::printf("scales %ld %ld\n", (long)M, (long)m0), 1;
            }
        }
  std::printf("ok %ld tiles, %ld of second launches\n", tiles, second);
  return second > 0 ? 0 : 2;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no C++ compiler")
def test_nothing_behind_the_operands(tmp_path):
    src, exe = tmp_path / "reach.cpp", tmp_path / "reach"
    # the two functions, out of a header that only a HIP compiler takes
    text = open(os.path.join(PKG, "csrc", "gemm_args.hpp")).read()
    reach = re.findall(r"__host__ __device__ (inline int64_t (?:tile|scale)_bytes\(.*?\n}\n)", text, flags=re.S)
    assert len(reach) == 2
    src.write_text(PROGRAM.replace("GEMM_REACH", "namespace puro {\n" + "".join(reach) + "}"))
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(PKG, "csrc"), str(src), "-o", str(exe),
                        "-L", PKG, "-lpuro_fp8", f"-Wl,-rpath,{PKG}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.startswith("ok"), f"exit {run.returncode}: {run.stdout} {run.stderr}"
