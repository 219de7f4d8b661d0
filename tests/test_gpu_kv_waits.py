"""Bounded waits of the wide draft-tree attention that run out at any point of the kernel."""
import pytest

from test_gpu_kv_attend import q8mv, wide  # noqa: F401

pytestmark = pytest.mark.gpu

# from the first wait of a CTA to longer than any
BOUNDS = [1, 300, 1000, 2000, 3000, 4000, 6000, 8000, 10000, 12000, 15000, 20000, 30000, 50000, 10 ** 6]


def again(c, first):
    """The same call has the bits of its first, checked answer, into memory that held none."""
    import torch

    got = c.run(out=torch.full_like(c.q, float("nan")))
    assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_a_plan_goes_on_whatever_the_bound_that_ran_out(q8mv):  # noqa: F811
    c = wide(q8mv, 21, [3000, 100, 9000], [40, 50, 33], heads=2, group=2, dim=128, dtype="bfloat16")
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
    c = wide(q8mv, 22, [3000, 100, 9000, 5], [40, 50, 33, 60], heads=2, group=2, dim=128, dtype="bfloat16")
    narrow = wide(q8mv, 23, [20000, 700], [3, 1], heads=2, group=2, dim=128, dtype="float32")
    narrow.plan = c.plan  # 16 rows at a time, with the same counters
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
