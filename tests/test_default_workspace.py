"""The MLP calls' own workspaces: what a captured graph holds stays allocated."""
import contextlib
import types
import weakref

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def sg(monkeypatch):
    import gemm_swiglu_mlp_gb300 as mod
    monkeypatch.setattr(mod, "_workspaces", {})
    monkeypatch.setattr(mod, "_outgrown", [], raising=False)
    return mod


@pytest.fixture
def cpu_streams(monkeypatch):
    """Streams without a GPU; returns whether each is being captured."""
    capturing, current = {}, [0]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream.cuda_stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing",
                        lambda: capturing.get(current[-1], False))
    return capturing


def test_outgrown_workspaces_stay_allocated(sg, cpu_streams):
    stream = types.SimpleNamespace(cuda_stream=7)
    first = sg._default_workspace("cpu", 100, stream)
    where, alive = first.data_ptr(), weakref.ref(first)
    del first
    second = sg._default_workspace("cpu", 101, stream)
    assert second.numel() >= 101 and second.data_ptr() != where and not second.any()
    assert alive() is not None
    # growing by a little each time does not add up
    for n in range(200, 5000, 50):
        last = sg._default_workspace("cpu", n, stream)
    assert sum(t.numel() for t in sg._outgrown) <= last.numel() <= 2 * 5000
    assert sg._default_workspace("cpu", 10, stream) is last


def test_no_workspace_is_made_on_a_stream_being_captured(sg, cpu_streams):
    """Whichever stream is current."""
    stream = types.SimpleNamespace(cuda_stream=7)
    cpu_streams[7] = True
    with pytest.raises(sg.SwigluError):
        sg._default_workspace("cpu", 100, stream)
    assert not sg._workspaces
    cpu_streams[7] = False
    ws = sg._default_workspace("cpu", 100, stream)
    cpu_streams[7] = True
    assert sg._default_workspace("cpu", 100, stream) is ws
    with pytest.raises(sg.SwigluError):
        sg._default_workspace("cpu", 101, stream)


@pytest.mark.gpu
def test_graph_survives_a_larger_call_on_its_stream():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gemm_swiglu_mlp_gb300 import build
    build.build()
    import gemm_swiglu_mlp_gb300 as sg
    cases = []
    for M, N, K in ((33, 264, 2000), (2048, 9728, 136)):
        A = torch.randn(M, K, device="cuda").bfloat16()
        W = [(torch.randn(K, N, device="cuda") * K ** -0.5).bfloat16() for _ in range(2)]
        cases.append((A, sg.swiglu_pack_weights(*W), N, sg.swiglu_workspace_bytes(M, N, K)))
    cases.sort(key=lambda c: c[3])
    (a, wp, n, need), (b, wpb, nb, more) = cases
    assert 0 < need < more
    want = sg.swiglu_up_forward(a, wp, n)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        sg.swiglu_up_forward(a, wp, n)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = sg.swiglu_up_forward(a, wp, n)
    with torch.cuda.stream(side):
        sg.swiglu_up_forward(b, wpb, nb)
        side.synchronize()
        fill = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
                for size in [need] * 8 + [1 << 20] * 32]
    torch.cuda.synchronize()
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((t == 0x5A).all()) for t in fill)
    assert sg.swiglu_check_device_status() == 0
