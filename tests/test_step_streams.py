"""With a given stream, whatever a call allocates is allocated as that stream's own: memory of the
current stream may still be in use there. Checked without a GPU on a stand-in for the native
calls, which only notes whether it runs on the stream or is handed it."""
import pytest

from gemm_swiglu_mlp_gb300 import cache, step

STREAM = object()


class Calls:
    """Every native call; a list of (ran on, handed)."""

    def __init__(self, monkeypatch):
        self.seen, self.on = [], None
        monkeypatch.setattr(cache, "_binding", self)
        monkeypatch.setattr(step, "_on", self.run_on)

    def run_on(self, stream, f, *args):
        self.on = stream
        try:
            return f(*args)
        finally:
            self.on = None

    def __getattr__(self, name):
        def call(*args):
            self.seen.append((self.on, args[-1]))
            return (1, 2, 3)
        return call


@pytest.mark.parametrize("out,allocates", [
    (None, True), (step.Verified(None, None, None), True), (step.Verified(1, None, None), True),
    (step.Verified(1, 2, None), True), (step.Verified(1, 2, 3), False)])
def test_verification(monkeypatch, out, allocates):
    calls = Calls(monkeypatch)
    step.swiglu_verify_drafts(0, 0, 0, width=1, out=out, stream=STREAM)
    step.swiglu_verify_drafts(0, 0, 0, width=1, out=out)
    assert calls.seen == [(STREAM, None) if allocates else (None, STREAM), (None, None)]


@pytest.mark.parametrize("q_out", [None, 1])
@pytest.mark.parametrize("k_out", [None, 1])
def test_rotation(monkeypatch, q_out, k_out):
    calls = Calls(monkeypatch)
    step.swiglu_head_rotate(0, 0, 0, q_out=q_out, k_out=k_out, stream=STREAM)
    step.swiglu_head_rotate_write(0, 0, 0, 0, 0, 0, 0, 0, q_out=q_out, stream=STREAM)
    assert calls.seen == [(None, STREAM) if q_out and k_out else (STREAM, None),
                          (None, STREAM) if q_out else (STREAM, None)]


@pytest.mark.parametrize("given", [None, 1])
def test_products(monkeypatch, given):
    # (a workspace may be allocated whatever is given)
    calls = Calls(monkeypatch)
    step.swiglu_up_forward_q4(0, 0, 0, 0, 0, Y=given, workspace=given, stream=STREAM)
    step.swiglu_down_forward_q4(0, 0, 0, out=given, workspace=given, stream=STREAM)
    step.swiglu_mlp_forward_q4(0, 0, 0, 0, 0, 0, 0, Y=given, out=given, workspace=given,
                               stream=STREAM)
    assert calls.seen == [(STREAM, None)] * 3
