"""How many CTAs a draft verification takes for a request, on the CPU (compiles
tests/verify_split_check.cpp): never a cluster larger than the device can run."""
import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "gemm_swiglu_mlp_gb300", "csrc")


def test_no_more_ctas_than_fit(tmp_path):
    exe = str(tmp_path / "verify_split_check")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + CSRC,
                    os.path.join(HERE, "verify_split_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout


def test_what_fits_is_asked_of_the_device():
    with open(os.path.join(CSRC, "step_api.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    setup = text[text.index("verify_setup_one("):text.index("int verify_device(")]
    assert "cudaOccupancyMaxActiveClusters" in setup
    call = text[text.index("int swiglu_verify_drafts("):text.index("swiglu_up_q4_workspace_bytes")]
    assert re.search(r"verify_ctas\([^;]*verify_cluster\)", call)
