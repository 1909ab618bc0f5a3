"""The recorded DRAM traffic of the fused kernels stands for their own sources only."""
import os
import shutil

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "gemm_swiglu_mlp_gb300", "csrc")


def test_hash_covers_the_fused_kernels_only(tmp_path):
    csrc = str(tmp_path / "csrc")
    shutil.copytree(CSRC, csrc)
    names = bench.fused_kernel_sources(csrc)
    assert names == sorted(["epilogue.cuh", "fused_up_kernel.cuh", "fused_up_pair_kernel.cuh",
                            "schedule.cuh", "sm103_ptx.cuh", "swiglu_api.cu"])
    before = bench.kernel_source_hash(csrc)
    assert before == bench.kernel_source_hash()
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name), "a") as f:
            f.write("// more\n")
        after = bench.kernel_source_hash(csrc)
        assert (after != before) == (name in names), name
        before = after
    with open(os.path.join(csrc, "another_kernel.cuh"), "w") as f:
        f.write("int x;\n")
    assert bench.kernel_source_hash(csrc) == before


@pytest.mark.parametrize("current", [True, False])
def test_traffic_is_reported_for_the_current_sources_only(tmp_path, monkeypatch, current):
    (tmp_path / "profiles").mkdir()
    (tmp_path / "profiles" / "traffic.json").write_text(
        '{"kernel_source_hash": "%s", "workloads": {"11": {"dram_bytes_per_launch": 5e9}}}'
        % (bench.kernel_source_hash() if current else "0" * 16))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.recorded_traffic("11") == (5e9 if current else None)
    assert bench.recorded_traffic("1") is None
