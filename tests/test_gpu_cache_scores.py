"""Attention scores far outside a model's range: finite scores of any size are
scores. A row is zero only if it sees nothing or nothing but scores of -inf."""
import numpy as np
import pytest

from tests import cache_ref as ref
from tests.test_gpu_cache import Case, sg  # noqa: F401  (the fixture)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def bits(x):
    return ref.f32_to_bits(np.array([x], np.float32))[0]


# Powers of two, so that scores are exact: D * 2^qe * 2^ke = 2^(qe + ke + 6) at D =
# 64, times the scale. One token is the narrow form, 40 of them the wide one.
@pytest.mark.parametrize("new", [1, 3, 40, 90])
@pytest.mark.parametrize("ctx", [20, 700])
@pytest.mark.parametrize("qe,ke,scale", [
    (50, 52, None), (60, 60, None),               # 2^105 and 2^123
    (50, 43, None), (50, 43, 0.123),              # 2^99, 6e29
    (10, 12, None), (11, 13, 0.3), (12, 13, 0.77),   # 2^25 to 2^31
    (14, 14, 0.77), (20, 20, 0.1), (1, 3, None),
    (30, 30, 1e-20), (60, 60, 1e-30), (-40, -40, 1e30)])
@pytest.mark.parametrize("sign", [-1, 1])
def test_finite_scores_of_any_size(sg, new, ctx, qe, ke, scale, sign):
    """Equal scores give the mean of the values, one larger score its value."""
    c = Case(new + ctx, [ctx, ctx + 9], [new, new], 7, 1, 64, 16, False)
    c.q[:] = bits(2.0 ** qe)
    used = c.k != 0x7FC0
    c.k[used] = bits(sign * 2.0 ** ke)
    c.check(c.run(sg, scale=scale), scale=scale)
    # the second request: some keys a unit in the last place above the others
    for x in (3, ctx // 2, ctx + 8):
        c.k[c.row(1, x)] = bits(sign * 2.0 ** ke * (1 + sign * 2.0 ** -7))
    c.check(c.run(sg, scale=scale), scale=scale)


@pytest.mark.parametrize("new", [1, 2, 40])
@pytest.mark.parametrize("mixed", [False, True])
def test_low_scores_beside_hidden_ones(sg, new, mixed):
    """Rows of very low finite scores and rows of ordinary ones in one group,
    after a first tile of nothing but -inf."""
    c = Case(3 + new, [400], [new], 8, 1, 64, 16, False)
    c.q[:] = bits(2.0 ** 50)
    if mixed:
        c.q[:, 1::2] = bits(2.0 ** -50)
    x = np.arange(400 + new)
    c.k[c.table[0, x // 16], :, x % 16] = bits(-2.0 ** 52)
    c.k[c.table[0, x[:300] // 16], :, x[:300] % 16] = 0xFF80
    c.check(c.run(sg))
