"""layer_norm of more rows than a launch takes at a time, for the widths up to 512 columns whose workgroups have several rows."""
import pytest
import torch

import allgather_gemm_amd as ag
from lm_reference import near
from test_lm_norm_gpu import BF16, EPS, backward, forward, gen, normal

pytestmark = pytest.mark.gpu

TURNS = [(40001, 100), (33000, 8), (20001, 200), (17000, 129), (9001, 500), (8200, 257)]


@pytest.mark.parametrize("rows,width", TURNS)
def test_rows_in_turn(rows, width):
    g = gen(rows + width)
    print("norm", rows, width, flush=True)
    x, res, w, b, dy = (normal(g, *s) for s in ((rows, width), (rows, width), (width,), (width,), (rows, width)))
    h = torch.empty_like(x)
    mean, rstd = torch.empty(2, rows, device="cuda")
    y = ag.layer_norm(x, weight=w, bias=b, eps=EPS, residual=res, h=h, mean=mean, rstd=rstd)
    s = (x.float() + res.float()).to(BF16)
    assert torch.equal(h, s)
    for name, got, (want, off) in zip(("y", "mean", "rstd"), (y, mean, rstd), forward(s, w, b, EPS)):
        near(got, want, off, name)
    for name, t, (want, off) in zip(("dx", "dw", "db"), ag.layer_norm_bwd(dy, h, mean, rstd, weight=w), backward(dy, h, mean, rstd, w, None)):
        near(t, want, off, name)
