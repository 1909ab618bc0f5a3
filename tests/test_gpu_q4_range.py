"""4-bit products at the ends of their range: tiny and huge rows and scales, values that are not
finite. Up to 8 rows sums are held in steps of 2^-76 (a group's before its scale, and the
result), and magnitudes of 2^67 and more are out of range; above 8 rows neither holds."""
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


def f64(t):
    return t.double().cpu().numpy()


def case(M, N, K, G, rows=1.0, scales=1.0):
    g = torch.Generator().manual_seed(M + N + G)
    A = (torch.randn(M, K, generator=g, dtype=torch.float64) * rows).bfloat16().cuda()
    Q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    S = ((torch.rand(K // G, N, generator=g, dtype=torch.float64) + 0.5) * (K ** -0.5 / 4 * scales)
         ).bfloat16().cuda()
    return A, Q, S


def check(sg, A, Q, S, G):
    """Within step_ref's bound, and: up to 8 rows each of a group's G / 16 matrix steps, and of those
    of the sum that it starts from, may be off by two steps, 2 * 2^-76 of the sum before the
    scale, G * 2^-78 in all; and the sums over the groups and shares by a step each. More
    rows: those sums have the units of BF16's own smallest step, 2^-133, or finer."""
    K, few = A.shape[1], A.shape[0] <= 8
    want, bound = ref.q4_down(f64(A), Q.cpu().numpy(), f64(S), G)
    if few:
        bound = bound + G * 2.0 ** -78 * np.abs(f64(S)).sum(0)
    bound = bound + (K / G + 17) * 2.0 ** (-76 if few else -133)
    got = f64(sg.swiglu_down_forward_q4(A, Q, S, group=G))
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], bound[bad][:4])
    return np.abs(want).mean(), bound.mean()


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 8, 9, 17])
@pytest.mark.parametrize("rows", [2.0 ** -60, 2.0 ** -64, 2.0 ** -70, 2.0 ** -100, 2.0 ** 64])
def test_tiny_and_huge_rows(sg, rows, M, G):
    size, bound = check(sg, *case(M, 136, 1280, G, rows=rows), G)
    if M > 8 or rows >= 2.0 ** -60:
        assert bound < size / 32        # (the bound says something)


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 8, 9, 17])
@pytest.mark.parametrize("scales", [2.0 ** -30, 2.0 ** -60, 2.0 ** -110, 2.0 ** 60])
def test_tiny_and_huge_scales(sg, scales, M, G):
    size, bound = check(sg, *case(M, 136, 1280, G, scales=scales), G)
    if M > 8 or scales >= 2.0 ** -60:
        assert bound < size / 32


def test_tiny_rows_share_a_line(sg):
    # more tiles than run at once: cut sums go through the workspace
    check(sg, *case(2, 24000, 4096, 128, rows=2.0 ** -60), 128)


@pytest.mark.parametrize("M", [1, 3, 8])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan"), 2.0 ** 72])
def test_values_out_of_range_reach_their_row_only(sg, M, value):
    G = 64
    A, Q, S = case(M, 136, 1280, G)
    want = sg.swiglu_down_forward_q4(A, Q, S, group=G)
    for k in (0, 1, 5, 700, 1279):
        B = A.clone()
        B[M - 1, k] = value
        got = sg.swiglu_down_forward_q4(B, Q, S, group=G)
        assert torch.isnan(got[M - 1]).all()
        assert torch.equal(got[:M - 1], want[:M - 1])
