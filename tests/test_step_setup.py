"""Draft verification and the 4-bit products set their kernels up at their own first call: the
setup that every call waits for, and fails with, has none of them; and a first call works
wherever it comes, in a capture too."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_common_setup_has_none_of_them():
    with open(os.path.join(ROOT, "gemm_swiglu_mlp_gb300", "csrc", "swiglu_api.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = text[text.index("int device_setup("):]
    body = body[:body.index("\n}\n")]
    assert "cudaFuncSetAttribute" in body and "down_decode_kernel" in body
    for name in ("verify", "q4", "rotate"):
        assert name not in body, name


FIRST = """
import sys, torch
sys.path.insert(0, %r)
import gemm_swiglu_mlp_gb300 as sg
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
tokens, start, u = i32([1, 2]), i32([0, 2]), torch.tensor([0.3, 0.9], device="cuda")
target = torch.zeros(2, 64000, device="cuda")
target[:, 50000] = 1.0
x = torch.ones(2, 512, dtype=torch.bfloat16, device="cuda")
codes = torch.full((64, 256), 0x99, dtype=torch.uint8, device="cuda")     # ones
scales = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
calls = {"verify": lambda: sg.swiglu_verify_drafts(tokens, start, target, uniform=u, width=2).next_tokens,
         "greedy": lambda: sg.swiglu_verify_drafts(tokens, start, i32_after, width=2).next_tokens,
         "product": lambda: sg.swiglu_down_forward_q4(x, codes, scales)}
i32_after = i32([2, 7])
want = {"verify": [50000], "greedy": [7], "product": [[512.0] * 64] * 2}
first, captured = sys.argv[1], sys.argv[2] == "captured"
for name in [first] + sorted(set(calls) - {first}):
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = calls[name]()
        graph.replay()
    else:
        got = calls[name]()
    assert got.tolist() == want[name], (name, got)
assert sg.swiglu_check_device_status() == 0
""" % ROOT


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["captured", "eager"])
@pytest.mark.parametrize("first", ["verify", "greedy", "product"])
def test_first_call_of_a_process(first, how):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_swiglu_mlp_gb300 import build
    build.build()
    run = subprocess.run([sys.executable, "-c", FIRST, first, how], capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0, run.stdout + run.stderr
