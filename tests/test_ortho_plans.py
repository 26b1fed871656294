"""Every way through newton_schulz's kernels that the plans choose for some extents is run by a test on the GPU."""
import os
import random

import pytest

import ortho_plans
import test_lm_ortho_gpu as shapes
import test_lm_ortho_ways_gpu as more

pytestmark = pytest.mark.skipif(not os.path.exists(ortho_plans.HIPCC), reason="hipcc not installed")


def extents():
    """Every 128th row count up to 9000 at five widths, wide and tall, and stacks."""
    for m in range(64, 9000, 128):
        for n in (m, m + 128, 2 * m, 3 * m, 4 * m):
            yield from ((1, m, n), (1, n, m))
    rng = random.Random(0)
    for _ in range(4000):
        yield (rng.choice([1, 1, 2, 3, 5, 8, 16, 32, 64]),) + tuple(int(2 ** rng.uniform(5, 13.5)) for _ in range(2))


def test_gpu_tests_take_every_way():
    taken = set()
    for stack in [(1,) + s for s in shapes.SHAPES + shapes.LARGE] + shapes.STACKS + more.WAYS:
        taken |= ortho_plans.ways(*stack)
    missing = {}
    for stack in extents():
        for way in ortho_plans.ways(*stack) - taken:
            missing.setdefault(way, stack)
    assert not missing


# X X^T, A A and B X, padded extents: the widest tiles and whether the last go in quarters, where that was the least of a sweep by more
# than a twentieth
SWEPT = [((1, 3200, 3200), "192", "192", "256"), ((1, 3328, 3328), "192", "192", "256"), ((1, 3456, 3456), "192", "192", "256"),
         ((1, 3968, 3968), "192", "192", "256"), ((1, 4352, 4352), "256", "256", "256q"), ((1, 4608, 4608), "256", "256", "256q"),
         ((1, 5760, 5760), "192", "192", "256q"), ((1, 6784, 6784), "256q", "256q", "256"), ((1, 7680, 7680), "256", "256", None),
         ((1, 8192, 8192), "256q", "256q", "256"), ((1, 2048, 5632), "128", "128", "256"), ((1, 3200, 6400), "192", "192", "256q"),
         ((9, 1280, 1280), "128", "128", "256"), ((10, 1024, 1024), None, None, "256"), ((28, 512, 512), "128q", "128q", "128")]


@pytest.mark.parametrize("stack,gram,square,update", SWEPT)
def test_plans_where_they_were_swept(stack, gram, square, update):
    got = ["%d%s" % (p.size, "q" if p.cut else "") for p in ortho_plans.plans(*stack)]
    assert [g for g, w in zip(got, (gram, square, update)) if w] == [w for w in (gram, square, update) if w]


def test_quarters_cost_rounds_of_their_own():
    """209 of 465 tiles in quarters are four rounds of them, 1.45 times the time of one of whole ones."""
    for E, m in ((1, 3840), (1, 3712), (1, 4608), (6, 1408), (9, 1280)):
        for p in ortho_plans.plans(E, m, m):
            if p.size == 128:
                assert p.cut == 0, (E, m, p)
