"""What the attention takes as a workspace of the caller's."""
import pytest

from tests.test_gpu_cache import Case, dev_bf16, dev_i32, host_bits, sg  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_workspace_checks(sg):
    c = Case(31, [300], [2], 4, 2, 64, 16, False)
    x = (dev_bf16(c.q), dev_bf16(c.k), dev_bf16(c.v), dev_i32(c.table), dev_i32(c.ctx),
         dev_i32(c.start))
    need = sg.swiglu_tree_attention_workspace_bytes(c.T, 4, 2, 64)
    strided = torch.zeros(2 * need, dtype=torch.uint8, device="cuda")[::2]
    assert strided.numel() >= need
    with pytest.raises(ValueError):
        sg.swiglu_tree_attention(*x, workspace=strided)
    with pytest.raises(TypeError):
        sg.swiglu_tree_attention(*x, workspace=torch.zeros(need, dtype=torch.uint8))
    with pytest.raises(TypeError):
        sg.swiglu_tree_attention(*x, workspace=need)
    whole = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")
    for bad in (whole[:need - 1], whole[16:need + 16]):     # too small; not aligned
        with pytest.raises(sg.SwigluError):
            sg.swiglu_tree_attention(*x, workspace=bad)
    # any type, of any content
    ok = torch.full((need // 4 + 1,), float("nan"), device="cuda")
    c.check(host_bits(sg.swiglu_tree_attention(*x, workspace=ok)))
