"""Draws whose numbers lie as near to a border as the contract speaks of: 2^-35 in rows whose
additions all round the same way, 2^-40 in rows of a softmax (held to about 2^-44). The borders
are exact: sums of whole numbers of 2^-62."""
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


def near_borders(row, distance, count):
    """`count` numbers j 2^-24 that fall nearest to a border of the FP32 row, though no nearer
    than `distance`, and the tokens they draw."""
    units = np.rint(row.astype(np.float64) * 2.0 ** 62).astype(np.int64)
    cdf = torch.from_numpy(np.cumsum(units)).cuda()
    total = int(cdf[-1])
    j = torch.arange(1 << 24, device="cuda")
    at = j * (total >> 24) + (j * (total & ((1 << 24) - 1)) >> 24)
    token = torch.searchsorted(cdf, at, right=True)
    before = torch.where(token > 0, cdf[(token - 1).clamp(min=0)], -(1 << 62))
    gap = torch.minimum(at - before, cdf[token] - at).double() * 2.0 ** -62
    gap[gap < distance] = 9.0
    nearest = torch.sort(gap).indices[:count]
    assert (gap[nearest] < 1).all()
    return (j[nearest].double() * 2.0 ** -24).float(), token[nearest], gap[nearest]


def peak(V):
    row = np.full(V, np.float32(0.45 / V), np.float32)
    row[5] = 0.55
    return row


def softmax(V):
    return ref.softmax_rows(np.random.default_rng(V), 1, V)[0]


# requests of one call: 1 and 8 CTAs each, 4, 1 and 16
@pytest.mark.parametrize("V,R", [(1 << 20, 160), (32000, 8), (128000, 64), (128000, 200),
                                 (1 << 20, 3)])
@pytest.mark.parametrize("make,distance", [(peak, 2.0 ** -35), (softmax, 2.0 ** -40)])
def test_numbers_beside_borders(sg, V, R, make, distance):
    row = make(V)
    target = torch.from_numpy(row).cuda().repeat(R, 1)
    start = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    tokens = torch.zeros(R, dtype=torch.int32, device="cuda")
    u, want, gap = near_borders(row, distance, max(R, 24) // R * R)
    assert gap.max() < 64 * distance
    for i in range(0, len(u), R):
        got = sg.swiglu_verify_drafts(tokens, start, target, uniform=u[i:i + R].contiguous(), width=1)
        bad = got.next_tokens.long() != want[i:i + R]
        assert not bad.any(), (int(bad.sum()), torch.log2(gap[i:i + R][bad])[:5])
