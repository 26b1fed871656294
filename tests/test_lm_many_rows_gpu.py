"""Cross entropies of more rows, and of more tiles, than one launch has workgroups for."""
import pytest
import torch

import allgather_gemm_amd as ag
import lm_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def check(T, K, V, rows):
    g = torch.Generator(device="cuda").manual_seed(T % 1000 + V)
    A = torch.randn(T, K, generator=g, device="cuda", dtype=BF16)
    B = torch.randn(V, K, generator=g, device="cuda", dtype=BF16)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y[::5] = -100
    print("xent", T, K, V, flush=True)
    loss, lse = ag.gemm_xent(A, B, y)
    for at in rows:
        (wl, ol), (ws, os_), _, _ = ref.xent(A[at], B, y[at])
        ref.near(loss[at], wl, ol, "loss %s" % (at,))
        ref.near(lse[at], ws, os_, "lse %s" % (at,))


def test_more_rows_than_a_launch_joins():
    n = 1 << 26                        # four rows a workgroup
    check(n + 5, 8, 8, [slice(0, 1 << 20), slice(n - (1 << 19), n + 5), slice(n // 2, n // 2 + 1000)])


def test_more_tiles_than_a_launch_has_workgroups():
    n = 1 << 21
    check(n + 1, 8, 1 << 17, [slice(0, 64), slice(n // 2 - 64, n // 2 + 64), slice(n - 300, n + 1)])
