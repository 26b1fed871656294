"""Sums over very many rows of layer_norm_bwd, against float64.

A column's terms pass at most rows / 8192 + 8 additions in a thread, where the rows are narrow, seven more in its workgroup and 128 + 8
where 1024 parts are joined; an fp32 sum of terms of one sign is off by at most that many times 2^-24, the result's rounding
by 2^-8."""
import pytest
import torch

import allgather_gemm_amd as ag
from lm_reference import F, H, near

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def additions(rows):
    return rows / 8192 + 160


@pytest.mark.parametrize("rows,width", [(1 << 27, 1), (1 << 25, 5)])
def test_terms_of_one_sign(rows, width):
    """1 + 2^-7 over and over: added one by one to more than 2^17 it is a sum of ones."""
    print("norm sums", rows, width, flush=True)
    dy = torch.full((rows, width), 1 + 2.0 ** -7, dtype=BF16, device="cuda")
    h = torch.ones_like(dy)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    _, dw, db = ag.layer_norm_bwd(dy, h, mean, rstd, need_dx=False)
    want = torch.full((width,), rows * (1 + 2.0 ** -7), dtype=torch.float64, device="cuda")
    for name, got in (("dw", dw), ("db", db)):
        near(got, want, want * (additions(rows) * F + H), name)


@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 6, 7])
def test_narrow_rows(width):
    rows = 300001 + 7 * width
    g = torch.Generator().manual_seed(width)
    dy = (torch.randn(rows, width, generator=g) + 0.5).to(BF16).cuda()
    h = torch.randn(rows, width, generator=g).to(BF16).cuda()
    mean, rstd = torch.randn(rows, generator=g).cuda(), torch.rand(rows, generator=g).cuda()
    _, dw, db = ag.layer_norm_bwd(dy, h, mean, rstd, need_dx=False)
    terms = dy.double() * (h.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for name, got, t in (("dw", dw, terms), ("db", db, dy.double())):
        off = (additions(rows) + 4) * F * t.abs().sum(0)
        near(got, t.sum(0), off * (1 + H) + H * t.sum(0).abs(), name)
    again = ag.layer_norm_bwd(dy, h, mean, rstd, need_dx=False)
    assert torch.equal(again[1], dw) and torch.equal(again[2], db)
