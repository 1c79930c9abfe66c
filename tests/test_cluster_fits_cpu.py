"""The size of a cluster where the device cannot place the largest one: a smaller one takes its place (whatever the
size, the sorted tokens are the same), never an error, and never less than every device can place."""
import os
import shutil
import subprocess

import pytest

from deterministic_token_logprob_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include "rlk_rows.cuh"
int main() {
  for (int most = 1; most <= 32; most *= 2) {
    int asked = 0;
    for (int want : {1, 2, 8, 16}) std::printf("%d ", rlk::cluster_that_fits(want, [&](int c) { ++asked; return c <= most; }));
    std::printf("%d\n", asked);
  }
  rlk::KnownPerDevice known;  // without a device there is no answer, and none is kept
  std::printf("%d\n", known([] { return 16; }));
}
"""


def test_cluster_that_fits(tmp_path):
    nvcc = build._nvcc()
    if not shutil.which(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "fits.cu", tmp_path / "fits"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, *build.ARCH, "-std=c++17", "-I", build.INCLUDE, "-I", build.CSRC, "-o", str(exe), str(src)],
                   check=True, capture_output=True)
    env = {**os.environ, "CUDA_VISIBLE_DEVICES": ""}
    lines = [list(map(int, x.split())) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True, env=env)
             .stdout.splitlines()]
    for most, got in zip((1, 2, 4, 8, 16, 32), lines):
        assert got == [1, 2, 8, 16 if most >= 16 else 8, 1], most
    assert lines[6] == [0]
