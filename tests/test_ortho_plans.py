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
