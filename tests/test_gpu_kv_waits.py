"""Bounded waits of the wide draft-tree attention that run out at any point of the kernel."""
import pytest

from test_gpu_kv_attend import q8mv, wide  # noqa: F401

pytestmark = pytest.mark.gpu

# from the first wait of a CTA to longer than any
BOUNDS = [1, 300, 1000, 2000, 3000, 4000, 6000, 8000, 10000, 12000, 15000, 20000, 30000, 50000, 10 ** 6]


def test_a_plan_goes_on_whatever_the_bound_that_ran_out(q8mv):  # noqa: F811
    c = wide(q8mv, 21, [3000, 100, 9000], [40, 50, 33], heads=2, group=2, dim=128, dtype="bfloat16")
    c.check()
    assert c.plan.check() == 0
    seen = set()
    for ns in BOUNDS:
        c.plan.set_wait(ns)
        c.run()
        seen.add(c.plan.check())
        c.plan.set_wait(0)
        c.check()
        assert c.plan.check() == 0
    assert seen == {0, 1}
