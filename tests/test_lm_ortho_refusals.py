"""Coefficients that newton_schulz refuses or takes by the extents, without a GPU."""
import ctypes

import pytest

import allgather_gemm_amd as ag

_vp = ctypes.c_void_p
P = [_vp(0x10000 + 0x1000 * i) for i in range(3)]      # never dereferenced: every call is refused


def taken(R, C, steps):
    """Whether the coefficients are: those that are fail at the workspace, which comes after them and is too small."""
    q = [x for abc in steps for x in abc]
    rc = ag.lib().newton_schulz(P[0], ag.TYPE_BF16, 1, R, C, (ctypes.c_float * len(q))(*q), len(steps), 1e-7, P[1], P[2], 0, None)
    assert rc in (ag.AG_EINVAL, ag.AG_EUNSUPPORTED)
    return rc == ag.AG_EINVAL


@pytest.mark.parametrize("steps,rows", [([(0.0, 1.0, 0.0)] * 2, 200), ([(0.0, 2.0, -1.0)] * 2, 300), ([(0.0, 0.0, 1.0)] * 2, 5),
                                        ([(0.0, 1.0, 0.0)] * 3, 6)])
def test_steps_that_leave_nothing(steps, rows):
    """Taken for up to some rows, refused from some more on: fp16 has few bits of A, B or X there."""
    assert all(taken(m, n, steps) for m in (1, 5, rows) for n in (m, 4 * m))
    assert not any(taken(m, n, steps) for m in (4 * rows, 4096, 1 << 16) for n in (m, 4 * m) if m * n <= 1 << 35)
    assert taken(4096, rows, steps) and not taken(1 << 16, 4096, steps)


@pytest.mark.parametrize("steps", [ag.NEWTON_SCHULZ, ag.NEWTON_SCHULZ * 4, [(1.5, -0.5, 0.0)] * 20, [(1.875, -1.25, 0.375)] * 10,
                                   [(2.0, -1.5, 0.5)] * 10, [(-1.0, 0.25, 0.0)] * 2, [(1.0, -1.0, 0.0)] * 3, [(0.0, 1.0, 0.0)],
                                   [(0.0, 0.0, 0.0)], [(1e-30, 0.0, 0.0)], [(0.02, 1.0, 0.0), (2.0, 0.0, 0.0)]])
def test_other_steps_are_taken_whatever_the_extents(steps):
    for R, C in ((1, 1), (1, 1 << 20), (1 << 20, 1), (64, 100), (4096, 4096), (14336, 4096), (1 << 17, 1 << 18)):
        assert taken(R, C, steps), (R, C)
