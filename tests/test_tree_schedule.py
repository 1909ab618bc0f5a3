"""Host-side check of the tree-attention work split (no GPU): compiles
tests/tree_schedule_check.cpp against tree_schedule.cuh and runs it over
random batches."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gemm_swiglu_mlp_gb300", "csrc")


def test_every_tile_once_and_shared_items_known(tmp_path):
    exe = str(tmp_path / "tree_schedule_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + CSRC,
                    os.path.join(HERE, "tree_schedule_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe, "600"], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout
