"""Bounded waits of the 128-row attention over the Q4_0 cache that run out, at any point of the kernel.

Only that kernel has waits, so a call whose wait ran out has reached it."""
import pytest

from test_gpu_kv4_attend import q8mv, wide  # noqa: F401
from test_gpu_kv_waits import BOUNDS, again

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 96, 128])
def test_a_plan_goes_on_whatever_the_bound_that_ran_out(q8mv, dim):  # noqa: F811
    c = wide(q8mv, 51, [3000, 100, 9000], [40, 50, 33], heads=2, group=2, dim=dim)
    first = c.run()
    c.check(first)
    assert c.plan.check() == 0
    seen = set()
    for ns in BOUNDS:
        c.plan.set_wait(ns)
        c.run()
        seen.add(c.plan.check())
        c.plan.set_wait(0)
        again(c, first)
        assert c.plan.check() == 0
    assert seen == {0, 1}


def test_a_wait_that_ran_out_spoils_its_own_call_alone(q8mv):  # noqa: F811
    """Nobody looks at the error word between the calls: the next one, of any shape, is right all the same."""
    c = wide(q8mv, 52, [3000, 100, 9000, 5], [40, 50, 33, 60], heads=2, group=2, dim=128)
    narrow = wide(q8mv, 53, [20000, 700], [3, 1], heads=2, group=2, dim=128)
    narrow.plan = c.plan  # 8 rows at a time, with the same counters
    first, first_narrow = c.run(), narrow.run()
    c.check(first), narrow.check(first_narrow)
    assert c.plan.check() == 0
    for ns in BOUNDS:
        for _ in range(3):
            c.plan.set_wait(ns)
            c.run()
            c.plan.set_wait(0)
            again(c, first)
            again(narrow, first_narrow)
    assert c.plan.check() == 1
    assert c.plan.check() == 0
