"""4-bit products whose every sum FP32 holds exactly: small whole numbers times codes, scales that are
powers of two. Then the result is the formula's, rounded once, bit for bit, at the longest sums:
any bit lost on the way shows."""
import numpy as np
import pytest

from tests import step_ref as ref

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


def case(M, N, K, G, seed, mats=1):
    """A of -2 .. 2, and weights of scales 2^-9 or 2^-8: K products of up to 2 * 8 * 2^-8 come to less
    than 2^24 steps of 2^-9 for K < 2^18."""
    g = torch.Generator().manual_seed(seed)
    A = torch.randint(-2, 3, (M, K), generator=g).bfloat16().cuda()
    w = []
    for _ in range(mats):
        w.append(torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda())
        w.append((2.0 ** torch.randint(-9, -7, (-(-K // G), N), generator=g)).bfloat16().cuda())
    return A, w


def product(A, codes, scales, G):
    """In 64 bits, on the GPU."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(1).double() - 8
    return A.double() @ (both * scales.double().repeat_interleave(G, 0)[:both.shape[1]].t()).t()


@pytest.mark.parametrize("M", [1, 5, 8, 9, 16, 17, 32, 40])
@pytest.mark.parametrize("N,K,G", [(64, 18944, 128), (136, 29568, 64), (200, 18976, 32),
                                   (1536, 29568, 128), (12008, 8224, 128)])
def test_plain(sg, M, N, K, G):
    A, (Q, S) = case(M, N, K, G, M + N)
    want = product(A, Q, S, G)
    assert float(want.abs().max()) < 2.0 ** 15      # (below 2^24 steps of 2^-9)
    assert torch.equal(sg.swiglu_down_forward_q4(A, Q, S, group=G), want.float().bfloat16())


@pytest.mark.parametrize("M", [1, 8, 9, 16, 17, 32])
@pytest.mark.parametrize("N,K,G", [(72, 18944, 128), (200, 29568, 64), (128, 18976, 32),
                                   (20232, 3584, 128)])
def test_gated(sg, M, N, K, G):
    """Exact sums through the FP32 activation (2^-18 of the result, as step_ref.q4_up has it) and one
    rounding."""
    A, (Q1, S1, Q2, S2) = case(M, N, K, G, M + N, mats=2)
    g, u = product(A, Q1, S1, G), product(A, Q2, S2, G)
    assert float(g.abs().max()) < 88
    want = g * torch.sigmoid(g) * u
    got = sg.swiglu_up_forward_q4(A, Q1, S1, Q2, S2, group=G)
    err = 2.0 ** -18 * want.abs()
    assert ((got.double() - want).abs() <= err + ref.BF16_U * (want.abs() + err)).all()


# a line of steps with cut tiles, shares of K on clusters, whole tiles; few rows and many
@pytest.mark.parametrize("M,N,K,gated", [(16, 12008, 4096, True), (1, 20232, 3584, True),
                                         (7, 24000, 2048, False), (1, 3584, 18944, False),
                                         (24, 512, 8192, False), (12, 2048, 2080, True)])
def test_the_same_from_run_to_run(sg, M, N, K, gated):
    """Again and again, captured, on two streams side by side: the same bits."""
    gen = torch.Generator().manual_seed(M)
    sets = []
    for _ in range(2):
        A = torch.randn(M, K, generator=gen).bfloat16().cuda()
        w = []
        for _ in range(2 if gated else 1):
            w.append(torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.uint8).cuda())
            w.append((torch.rand(-(-K // 128), N, generator=gen) + 0.5).bfloat16().cuda() * K ** -0.5)
        sets.append((A, w))
    call = sg.swiglu_up_forward_q4 if gated else sg.swiglu_down_forward_q4
    want = [call(A, *w) for A, w in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for i in range(40):
        for (A, w), s in zip(sets, streams):
            got.append(call(A, *w, stream=s))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [call(A, *w) for A, w in sets]
    for _ in range(20):
        for y in captured:
            y.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(y, z) for y, z in zip(captured, want))
    assert sg.swiglu_check_device_status() == 0
