"""Every device function of the sources is called by something."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "gemm_swiglu_mlp_gb300", "csrc")


def test_every_device_function_has_a_caller():
    text = ""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text += re.sub(r"//[^\n]*", "", f.read()) + "\n"
    names = set(re.findall(r"(?:__device__|__forceinline__|__noinline__|SWIGLU_HD|SWIGLU_HD_CALL)\s+"
                           r"(?:static\s+)?[\w:<>, ]+?[\s*&]+(\w+)\(", text))
    assert len(names) > 100
    unused = [n for n in sorted(names) if len(re.findall(r"\b%s\b" % n, text)) < 2]
    assert not unused, unused
