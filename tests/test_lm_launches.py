"""The launches of the language-model operators, recorded on the host (lm_launches.py): their sizes."""
import os

import pytest

import lm_launches as lm

pytestmark = pytest.mark.skipif(not os.path.exists(lm.HIPCC), reason="hipcc not installed")

MOST_ROWS, MOST_COLUMNS = 1 << 30, 1 << 21
# the largest extents that the entry points take, in each direction, and some that a card's memory holds
EXTREME_XENT = [(MOST_ROWS, 8, 1), (MOST_ROWS, 8, 128), (1 << 26, 8, 8), (1 << 24, 8, 32769), ((1 << 21) + 1, 8, 1 << 17),
                (1 << 14, MOST_COLUMNS, 512), (1, 8, MOST_COLUMNS), (1 << 12, 64, MOST_COLUMNS), (3, MOST_COLUMNS, 3)]
EXTREME_LINEAR = [(MOST_ROWS, 8, 1), (1 << 24, 8, 1 << 10), (1 << 24, 128, 1 << 14), (1, MOST_COLUMNS, MOST_COLUMNS),
                  (64, 8, MOST_COLUMNS), (1 << 14, 64, MOST_COLUMNS), (1 << 14, MOST_COLUMNS, 64)]


def fits(launches):
    assert launches
    for l in launches:
        # the runtime counts the threads along x in 32 bits, workgroups along y and z in 16
        assert 1 <= l.grid[0] and l.grid[0] * l.block[0] < 1 << 32, l
        assert 1 <= l.grid[1] < 1 << 16 and l.grid[2] == 1, l


@pytest.mark.parametrize("shape", EXTREME_XENT)
def test_launches_of_the_largest_cross_entropies_are_valid(shape):
    fits(lm.xent(*shape))
    fits(lm.xent_bwd(*shape))
    T, K, V = shape
    least = T * 512 + (T + 64) * K * 4 * 64 + (1 << 20)
    fits(lm.xent_bwd(T, K, V, work_bytes=least))


@pytest.mark.parametrize("shape", EXTREME_LINEAR)
def test_launches_of_the_largest_linear_layers_are_valid(shape):
    M, K, Nc = shape
    fits(lm.linear(M, K, Nc))
    fits(lm.linear(M, K, Nc, "silu", True, True, True))
    fits(lm.linear_bwd(M, K, Nc, "gelu"))


@pytest.mark.parametrize("shape", [(1024, 1 << 15, 64, 64), (1024, 1, 8, MOST_COLUMNS), (1, MOST_ROWS, 8, 8), (1, 1, 1 << 14, 1 << 14),
                                   (1024, 1 << 24, 64, 1 << 10)])
def test_launches_of_the_largest_grouped_products_are_valid(shape):
    fits(lm.grouped(*shape))
    fits(lm.grouped_bwd(*shape))


def test_slices_of_a_join_cover_its_rows():
    """Rows past a launch's limit go to another one, and no row to two."""
    T = MOST_ROWS
    joins = [l for l in lm.xent(T, 8, 1) if l.kernel == "xent_join<1>"]
    assert len(joins) > 1 and sum(l.grid[0] for l in joins) == T // 4
    joins = [l for l in lm.xent(1 << 24, 8, 32769) if l.kernel == "xent_join<4>"]
    assert len(joins) > 1 and sum(l.grid[0] for l in joins) == 1 << 24
