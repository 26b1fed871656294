"""Every kernel of layer_norm and its gradients is run by the GPU's tests with exactly the extents and arguments that these have,
once a row each and once with more rows than a launch takes at a time."""
import os

import pytest

import norm_ortho_launches as launches
import test_lm_norm_gpu as norm_tests
from test_lm_norm_turns_gpu import TURNS

pytestmark = pytest.mark.skipif(not os.path.exists(launches.HIPCC), reason="hipcc not installed")


def norm_kernels():
    return {k for k in launches.kernels() if k.startswith("norm_")} | {k for k in launches.kernels() if k.startswith("norm<")}


def of_widths():
    """test_forward_and_backward: three row counts for each width, with dh for two widths of three."""
    for i, width in enumerate(norm_tests.WIDTHS):
        for rows in (norm_tests.ROWS[i % 9], norm_tests.ROWS[(i * 4 + 3) % 9], 1):
            yield launches.norm(rows, width)
            for args in (dict(), dict(sums=False), dict(dx=False)):
                yield launches.norm_bwd(rows, width, dh=bool(i % 3), **args)


def of_many_rows():
    """test_many_rows: with and without dh."""
    for rows, width in norm_tests.MANY:
        yield launches.norm(rows, width)
        for dh in (False, True):
            yield launches.norm_bwd(rows, width, dh=dh)


def test_every_kernel_is_run():
    seen = {l.kernel for call in of_widths() for l in call} | {l.kernel for call in of_many_rows() for l in call}
    assert norm_kernels() <= seen, norm_kernels() - seen


def test_rows_in_turn():
    """The kernels that go over rows by turns do so in one of the tests."""
    turns = set()
    for rows, width in norm_tests.MANY + TURNS:
        for l in (launches.norm(rows, width) + launches.norm_bwd(rows, width) + launches.norm_bwd(rows, width, dh=False)):
            args = [int(x) for x in l.kernel.split("<")[1][:-1].split(",")] if "<" in l.kernel else [1024]
            if l.grid[0] * max(1, l.block[0] // args[0]) < rows:
                turns.add(l.kernel)
    once = {k for k in norm_kernels() if "few" in k or "cols" in k or "join" in k}     # a row each, or by columns
    assert norm_kernels() - once <= turns, norm_kernels() - once - turns
