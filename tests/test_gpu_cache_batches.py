"""Attention of batches as a server has them: more requests than the kernel's blocks
have threads, single tokens beside trees, whole prompts."""
import numpy as np
import pytest

from tests.test_gpu_cache import Case, sg  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [640, 641, 700, 1500])
@pytest.mark.parametrize("tree", [False, True])
def test_more_requests_than_threads(sg, R, tree):
    """Requests of one token, of some and of more rows than the narrow form takes,
    and without any, in runs and mixed."""
    rng = np.random.default_rng(R + tree)
    ctx = np.where(rng.random(R) < 0.03, rng.integers(500, 3000, R), rng.integers(0, 150, R))
    new = rng.choice([0, 1, 3, 11, 40], R, p=[0.2, 0.5, 0.2, 0.07, 0.03])
    new[100:300] = 1
    new[300:330] = 0
    new[-3:] = 0, 9, 0
    c = Case(R, ctx, new, 4, 1, 64, 16, tree)
    c.check(c.run(sg))


@pytest.mark.parametrize("Hq,Hkv,D,P", [(7, 1, 128, 16), (8, 2, 64, 64)])
def test_single_tokens_beside_trees(sg, Hq, Hkv, D, P):
    """Both forms with work of their own, every other request of each."""
    rng = np.random.default_rng(D)
    ctx = rng.integers(1, 1200, 48)
    new = np.where(np.arange(48) % 2, rng.integers(20, 65, 48), 1)
    c = Case(D + 1, ctx, new, Hq, Hkv, D, P, True)
    c.check(c.run(sg))


@pytest.mark.parametrize("ctx,new,Hq,Hkv,D,P", [
    ([0], [2500], 2, 1, 128, 16),
    ([0, 0, 37], [1100, 2049, 1], 3, 1, 64, 64),
    ([0, 130], [4097, 300], 1, 1, 64, 128),
])
def test_whole_prompts(sg, ctx, new, Hq, Hkv, D, P):
    c = Case(sum(new), ctx, new, Hq, Hkv, D, P, False)
    c.check(c.run(sg))
