"""Plans whose buffers are used again, fed with what the step before left."""
import numpy as np
import pytest

from tests import cache_ref as ref
from tests.test_gpu_cache import dev_i32, sg  # noqa: F401

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_two_plans_alternate(sg):
    """Six steps, each with the pages and the free list's head of the plan before,
    in the buffers of the one before that."""
    rng = np.random.default_rng(41)
    R, P, width, pages = 6, 16, 20, 80
    free = rng.permutation(pages)
    table = np.full((R, 12), -1, np.int64)
    tab, dev_free = dev_i32(table), dev_i32(free)
    ctx, held, head = np.zeros(R, np.int64), np.zeros(R, np.int64), 0
    plans = [None, None]
    dev_held, dev_head = dev_i32(held), None
    for step in range(6):
        new = rng.integers(0, width + 1, R)
        par = np.stack([ref.random_parents(rng, width) for _ in range(R)])
        buffers = plans[step % 2]
        got = sg.swiglu_cache_plan(dev_i32(ctx), dev_i32(new), dev_held, tab, dev_free, P, R * width,
                                   parents=dev_i32(par), free_head=dev_head, out=buffers)
        assert buffers is None or got.slots.data_ptr() == buffers.slots.data_ptr()
        want = ref.plan(ctx, new, held, table, free, P, R * width, par, head)
        for name in ("query_start", "slots", "positions", "pages_held", "counts", "mask"):
            assert np.array_equal(getattr(got, name).cpu().numpy(), want[name]), (step, name)
        assert np.array_equal(tab.cpu().numpy(), want["table"])
        plans[step % 2] = got
        dev_held, dev_head = got.pages_held, got.counts[2:3]
        ctx, held, head = ctx + new, want["pages_held"], int(want["counts"][2])
    assert head == (-(-ctx // P)).sum()


def test_a_plan_does_not_take_its_own_outputs(sg):
    ctx, new, held = dev_i32([3, 20]), dev_i32([2, 1]), dev_i32([1, 2])
    table, free = dev_i32([[0, -1, -1], [1, 2, -1]]), dev_i32([5, 6, 7])
    first = sg.swiglu_cache_plan(ctx, new, held, table, free, 16, 4)
    before = [t.clone() for t in first if t is not None]
    for kw in (dict(free_head=first.counts[2:3]), dict(held=first.pages_held)):
        x = dict(dict(held=held, free_head=None), **kw)
        with pytest.raises(sg.SwigluError):
            sg.swiglu_cache_plan(ctx, new, x["held"], table, free, 16, 4, free_head=x["free_head"],
                                 out=first)
    assert all(torch.equal(a, b) for a, b in zip(before, first))
