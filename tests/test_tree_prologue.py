"""Host-side check of how the attention kernel's blocks find their start (no GPU):
compiles tests/tree_prologue_check.cpp against tree_schedule.cuh, with batches of
more requests than the kernel has threads among its cases."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gemm_swiglu_mlp_gb300", "csrc")


def test_every_block_finds_its_start(tmp_path):
    exe = str(tmp_path / "tree_prologue_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I" + CSRC,
                    os.path.join(HERE, "tree_prologue_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe, "150"], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout
