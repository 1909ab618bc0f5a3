"""The three results of a draft verification are tensors of their own: what a caller does to one
(resizing it for another tree, reusing it as `out`) leaves the others as they are."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_swiglu_mlp_gb300 import build
    build.build()
    import gemm_swiglu_mlp_gb300 as mod
    torch.cuda.set_device(0)
    return mod


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def greedy(sg, **kw):
    # two chains of two; the first holds, the second does not
    return sg.swiglu_verify_drafts(i32([1, 2, 3, 4]), i32([0, 2, 4]), i32([2, 9, 5, 7]), width=2, **kw)


def test_resizing_one_leaves_the_others(sg):
    for name in ("paths", "path_lens", "next_tokens"):
        got = greedy(sg)
        assert got.paths.tolist() == [[0, 1], [0, -1]]
        assert got.path_lens.tolist() == [2, 1] and got.next_tokens.tolist() == [9, 5]
        kept = {n: getattr(got, n).clone() for n in got._fields if n != name}
        getattr(got, name).resize_(2, 3).fill_(77)
        for n, want in kept.items():
            assert torch.equal(getattr(got, n), want), (name, n)


def test_no_shared_memory(sg):
    got = greedy(sg)
    starts = {t.untyped_storage().data_ptr() for t in got}
    assert len(starts) == 3 and all(t.is_contiguous() and t.storage_offset() == 0 for t in got)
    assert all(t.device == torch.device("cuda:0") and t.dtype == torch.int32 for t in got)
    for t in got:                        # known to the allocator as any other tensor is
        t.record_stream(torch.cuda.Stream())


def test_without_requests(sg):
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    got = sg.swiglu_verify_drafts(e, i32([0]), e, width=3)
    assert got.paths.shape == (0, 3) and got.path_lens.shape == got.next_tokens.shape == (0,)


def test_in_a_captured_call(sg):
    args = [i32([1, 2, 3, 4]), i32([0, 2, 4]), i32([2, 9, 5, 7])]
    sg.swiglu_verify_drafts(*args, width=2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sg.swiglu_verify_drafts(*args, width=2)
    args[2].copy_(i32([9, 1, 4, 8]))
    graph.replay()
    assert got.paths.tolist() == [[0, -1], [0, 1]]
    assert got.path_lens.tolist() == [1, 2] and got.next_tokens.tolist() == [9, 8]
