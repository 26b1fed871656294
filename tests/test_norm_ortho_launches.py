"""The plans of layer_norm, its gradients and newton_schulz without a GPU: the shapes of the GPU tests reach every kernel that
the library has, launches stay within what HIP counts, and the shapes that the plans were measured on go where they were
fastest."""
import os

import pytest

import norm_ortho_launches as launches
import test_lm_norm_gpu as norm_tests
import test_lm_ortho_gpu as ortho_tests

pytestmark = pytest.mark.skipif(not os.path.exists(launches.HIPCC), reason="hipcc not installed")


def ortho_shapes():
    for R, C in ortho_tests.SHAPES:
        yield 1, R, C, False
        yield 1, R, C, True
    for R, C in ortho_tests.LARGE:
        yield 1, R, C, True
    for E, R, C in ortho_tests.STACKS:
        yield E, R, C, False


def test_gpu_tests_reach_every_kernel():
    seen = set()
    for rows in norm_tests.ROWS:
        for width in norm_tests.WIDTHS:
            seen |= {l.kernel for l in launches.norm(rows, width)}
            for dh in (False, True):
                seen |= {l.kernel for l in launches.norm_bwd(rows, width, dh=dh)}
    for rows, width in norm_tests.MANY:
        for dh in (False, True):
            seen |= {l.kernel for l in launches.norm_bwd(rows, width, dh=dh)}
    for shape in ortho_shapes():
        seen |= {l.kernel for l in launches.schulz(*shape)}
    assert launches.kernels() == seen, launches.kernels() ^ seen


@pytest.mark.parametrize("call", [lambda: launches.norm(1 << 30, 8), lambda: launches.norm(1 << 30, 1 << 21),
                                  lambda: launches.norm_bwd(1 << 30, 8), lambda: launches.norm_bwd(1 << 30, 1 << 21),
                                  lambda: launches.norm_bwd(5, 1 << 21), lambda: launches.schulz(65535, 1, 1),
                                  lambda: launches.schulz(1, 1 << 20, 256), lambda: launches.schulz(1, 1 << 20, 250, True),
                                  lambda: launches.schulz(1, 1 << 18, 1 << 17), lambda: launches.schulz(60000, 1024, 1024),
                                  lambda: launches.schulz(30000, 256, 4096), lambda: launches.schulz(65535, 130, 120),
                                  lambda: launches.schulz(1024, 8192, 8192)])
def test_launches_of_the_largest_calls(call):
    """HIP counts a launch's threads along x in 32 bits, and workgroups along y and z in 16."""
    for l in call():
        assert 0 < l.grid[0] and l.grid[0] * l.block[0] < 1 << 32, l
        assert 0 < l.grid[1] <= 65535 and 0 < l.grid[2] <= 65535, l
        assert l.block[0] <= 1024 and l.block[1:] == (1, 1), l


def names(E, m, n):
    """Kernels of a step's products."""
    return tuple(l.kernel for l in launches.schulz(E, m, n)[2:] if l.kernel.startswith("ortho"))[:3]


@pytest.mark.parametrize("shape,want", [
    ((1, 512, 1024), ("ortho64<5,2,0>", "ortho64<6,2,0>", "ortho64<7,2,0>")),
    ((1, 1024, 4096), ("ortho64<5,2,0>", "ortho64<6,2,0>", "ortho128<7>")),
    ((1, 2048, 2048), ("ortho128<5>", "ortho128<6>", "ortho128<7>")),
    ((1, 4096, 4096), ("ortho192<5>", "ortho192<6>", "ortho256<7>")),
    ((16, 1024, 2048), ("ortho128<5>", "ortho128<6>", "ortho256<7>")),
    ((1, 6016, 6016), ("ortho256<5>", "ortho256<6>", "ortho256<7>")),
    ((1, 250, 8000), ("ortho64<5,2,1>", "ortho_thin<256>", "ortho64<5,2,1>")),
    ((1, 100, 5440), ("ortho64<5,2,1>", "ortho_thin<128>", "ortho64<5,2,1>"))])
def test_plans_where_they_were_measured(shape, want):
    assert names(*shape) == want


def test_workspace_is_what_the_steps_hold():
    """Three copies of X, two of A, sums of squares and, where a reduction goes in parts, at most two fp32 tiles for a CU."""
    L = launches.recorder()
    for E, R, C in ((1, 1, 1), (1, 4096, 4096), (7, 300, 5000), (1, 100, 8000), (16, 2048, 1024), (1, 1 << 20, 64)):
        mp, np = -(-min(R, C) // 128) * 128, -(-max(R, C) // 128) * 128
        least = E * (6 * mp * np + 4 * mp * mp)
        n = L.newton_schulz_workspace(E, R, C)
        assert least <= n <= least + E * (8 * 1024 + 8) + 9 * 256 + 2 * 512 * 32768, (E, R, C)
