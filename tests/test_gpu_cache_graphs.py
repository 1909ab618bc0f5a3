"""Captured attention calls that bring no workspace of their own: a graph owns the
memory that its replays write."""
import numpy as np
import pytest

from tests.test_gpu_cache import Case, dev_bf16, dev_i32, dev_i64, host_bits, sg  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def inputs(c):
    m = c.mask()
    return (dev_bf16(c.q), dev_bf16(c.k), dev_bf16(c.v), dev_i32(c.table), dev_i32(c.ctx),
            dev_i32(c.start), None if m is None else dev_i64(m))


def small_and_large():
    """One row tile a request at head size 64; two at 128, whose workspace is four
    times as large. Long contexts, so that items are shared between blocks."""
    return (Case(21, [6000, 900], [9, 3], 7, 1, 64, 16, True),
            Case(22, [5000, 900], [40, 30], 7, 1, 128, 16, True))


def test_graph_survives_a_larger_call_on_its_stream(sg):
    """Warm up and capture a small call, let a larger one grow the stream's
    workspace, hand all free memory out again, replay."""
    small, large = small_and_large()
    a, b = inputs(small), inputs(large)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        sg.swiglu_tree_attention(*a)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = sg.swiglu_tree_attention(*a)
    with torch.cuda.stream(side):
        big = sg.swiglu_tree_attention(*b)
        side.synchronize()
        # blocks of the old workspace's size and of others, from the stream's pool
        need = sg.swiglu_tree_attention_workspace_bytes(small.T, 7, 1, 64)
        fill = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
                for n in [need] * 4 + [1 << 20] * 64 + [1 << 16] * 64]
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        small.check(host_bits(out))
    assert all(bool((t == 0x5A).all()) for t in fill)
    large.check(host_bits(big))
    assert sg.swiglu_check_device_status() == 0


@pytest.mark.parametrize("given", ["current", "stream", "stream and out"])
def test_capture_needs_no_warm_up(sg, given):
    """The first call of a stream may be a captured one, with the stream current
    or given, and two graphs of one stream replay at the same time as its calls."""
    small, large = small_and_large()
    graphs = []
    side = torch.cuda.Stream()
    for c in (small, large):
        x = inputs(c)
        out = torch.empty_like(x[0])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            if given == "current":
                got = sg.swiglu_tree_attention(*x)
            elif given == "stream":
                got = sg.swiglu_tree_attention(*x, stream=side)
            else:
                # (on a forked stream that the capture takes in)
                fork = torch.cuda.Stream()
                fork.wait_stream(side)
                got = sg.swiglu_tree_attention(*x, out=out, stream=fork)
                side.wait_stream(fork)
        graphs.append((c, x, g, got))
    others = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    eager = []
    for _ in range(5):
        for s, (c, x, g, got) in zip(others, graphs):
            with torch.cuda.stream(s):
                g.replay()
        for c, x, _, _ in graphs:
            eager.append((c, sg.swiglu_tree_attention(*x, stream=side)))
    torch.cuda.synchronize()
    for c, _, _, got in graphs:
        c.check(host_bits(got))
    for c, got in eager[-2:]:
        c.check(host_bits(got))
    for i, (_, got) in enumerate(eager):
        assert torch.equal(got, eager[i % 2][1])
    assert sg.swiglu_check_device_status() == 0


def test_capture_of_several_calls(sg):
    """Calls one after the other in one graph, as the layers of a step are."""
    small, large = small_and_large()
    a, b = inputs(small), inputs(large)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [sg.swiglu_tree_attention(*x) for x in (a, b, a, b, b)]
    g.replay()
    torch.cuda.synchronize()
    for c, out in zip((small, large, small, large, large), outs):
        c.check(host_bits(out))


def test_default_workspace_grows_between_calls(sg):
    """Two sizes on one stream, back to back without a wait between them."""
    small, large = small_and_large()
    a, b = inputs(small), inputs(large)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = [sg.swiglu_tree_attention(*x) for x in (a, b, a, b)]
    side.synchronize()
    for c, out in zip((small, large) * 2, got):
        c.check(host_bits(out))
    assert np.array_equal(host_bits(got[0]), host_bits(got[2]))
