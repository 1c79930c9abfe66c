"""The committed traffic record serves as long as the tile kernels' sources are those that it was taken from,
whatever else the library holds."""
import os
import shutil

import bench
from deterministic_token_logprob_gb300 import build


def test_committed_record_serves_the_tile_kernels_of_this_tree():
    for stage in ("fwd", "dz", "dH", "dW"):
        value, note = bench.traffic_per_launch(stage)
        assert value and value > 1e9, note


def test_hash_follows_the_tile_kernels_alone(tmp_path, monkeypatch):
    shutil.copytree(build.CSRC, tmp_path / "csrc")
    monkeypatch.setattr(build, "CSRC", str(tmp_path / "csrc"))
    before = build.tile_kernel_sources_sha256()
    touched = {f for f in os.listdir(tmp_path / "csrc")}
    changes = set()
    for name in sorted(touched):
        p = tmp_path / "csrc" / name
        text = p.read_text()
        p.write_text(text + "// more\n")
        if build.tile_kernel_sources_sha256() != before:
            changes.add(name)
        p.write_text(text)
    assert changes == {"rlk_api.cu", "rlk_gemm.cuh", "rlk_gemm_fwd.cu", "rlk_gemm_dz.cu", "rlk_gemm_dh.cu",
                       "rlk_gemm_dw.cu", "rlk_ptx.cuh", "rlk_internal.h"}
