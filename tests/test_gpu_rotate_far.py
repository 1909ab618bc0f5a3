"""Rotation at far positions and by fast frequencies, to the accuracy of the contract: angles within
2^-26 turns and |inv_freq * position| 2^-64. Exact angles by whole numbers: an FP32 frequency is
m 2^-e, and pi is taken to 200 bits."""
from fractions import Fraction

import numpy as np
import pytest

from tests import step_ref as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)


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


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_angles_at_any_position(sg, D, interleaved):
    g = torch.Generator().manual_seed(D)
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 10 ** 9 + 7, 123456789, -987654321, 4097]
    pos += torch.randint(-2 ** 31, 2 ** 31, (40,), generator=g).tolist()
    freq = [1.0, 0.5, 1e-3, 1e-7, 3.0, 100.0, -0.25, 1e-40, 0.75, 2.0 ** -12, 6.2831855, -99.5,
            1.1754944e-38, 1e-5, 0.1, 31.0]
    f = torch.tensor(freq, device="cuda")
    n, T = len(freq), len(pos)
    q = torch.randn(T, 2, D, generator=g).bfloat16().cuda()
    k = torch.randn(T, 1, D, generator=g).bfloat16().cuda()
    qo, ko = sg.swiglu_head_rotate(q, k, torch.tensor(pos, dtype=torch.int32, device="cuda"), f,
                                   interleaved=interleaved)
    values = [Fraction(v) for v in f.tolist()]
    angle = np.array([[float((v * p) % (2 * PI)) for v in values] for p in pos])[:, None]
    far = np.abs(np.array(pos, np.float64)[:, None] * np.array(f.tolist()))[:, None]
    # the angle as stated, one unit in 2^-32 turns that is cut off, a truncated frequency's
    # unit of 2^-64 turns times the position (2^-33); sine and cosine (2^-23), two products and
    # a sum (2^-24 each) come to 2^-22; and one rounding to BF16
    off = 2 * np.pi * (2.0 ** -26 + far * 2.0 ** -64 + 2.0 ** -32 + 2.0 ** -33) + 2.0 ** -22
    one, two = ((slice(0, n), slice(n, 2 * n)) if not interleaved
                else (slice(0, 2 * n, 2), slice(1, 2 * n, 2)))
    c, s = np.cos(angle), np.sin(angle)
    for got, x in ((qo, q), (ko, k)):
        a, b = f64(x)[..., one], f64(x)[..., two]
        for part, want in ((one, a * c - b * s), (two, a * s + b * c)):
            err = off * (np.abs(a) + np.abs(b))
            bad = ~(np.abs(f64(got)[..., part] - want) <= err + ref.BF16_U * (np.abs(want) + err))
            assert not bad.any(), np.argwhere(bad)[:5]
        assert torch.equal(got[..., 2 * n:], x[..., 2 * n:])
