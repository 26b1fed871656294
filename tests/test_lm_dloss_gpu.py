"""The cross entropy's gradients for one dloss at all rows (a mean's 1 / n), against float64 and element by element: with the
d logits counted in units of it, what is rounded to bf16 is softmax - 1 at a row's target.  That is off by at most half a
step, H (1 - p), and by at most p, for -1 is a bf16 value; the other d logits by H p.  Rounded as dloss (softmax - 1), every
row would be off by as much of dloss as dloss itself, up to H."""
import pytest
import torch

import allgather_gemm_amd as ag
import lm_reference as ref
from lm_reference import E, F, H
from test_lm_kernels_gpu import xent_inputs

pytestmark = pytest.mark.gpu

# as far from a bf16 value as there is, a third, two numbers of tokens, a large and a small scale
DLOSS = [1 + 2.0 ** -8, 1 / 3, 1 / 253, -1 / 3796, 2.0 ** 20 / 3, 2.0 ** -30 / 3]


def common_dloss(w, A, B, y, lse):
    """((dA, bound), (dB, bound)) for w of one value and zeros: lm_reference.xent_bwd with the roundings named above."""
    a, b, g = A.double(), B.double(), w.double().unsqueeze(1)
    z, off = ref.product(a, b)
    has = ((y >= 0) & (y < B.shape[0])).unsqueeze(1)
    g = torch.where(has, g, torch.zeros_like(g))
    hit = torch.zeros_like(z).scatter_(1, torch.where(has, y.unsqueeze(1), 0), 1.0)
    p = torch.exp(z - lse.double().unsqueeze(1))
    p_off = p * (torch.expm1(off + F * lse.double().abs().unsqueeze(1)) + E) + 4 * F
    D = (p - hit) * g
    rounded = torch.where(hit > 0, torch.minimum(p, H * (1 - p).abs()), H * p)
    D_off = (p_off * (1 + H) + rounded) * g.abs()
    dA, offA = ref.product(D, b.t().contiguous())
    dB, offB = ref.product(D.t().contiguous(), a.t().contiguous())
    offA = offA * (1 + H) + D_off @ b.abs()
    offB = offB * (1 + H) + D_off.t() @ a.abs()
    return (dA, offA * (1 + H) + H * dA.abs()), (dB, offB * (1 + H) + H * dB.abs())


@pytest.mark.parametrize("shape", [(20, 1024, 1003), (60, 512, 3001), (300, 512, 2049), (2300, 264, 4099), (4353, 1000, 4090)])
@pytest.mark.parametrize("dloss", DLOSS)
def test_a_dloss_common_to_all_rows_is_not_rounded(shape, dloss):
    T, K, V = shape
    print("xent", shape, dloss, flush=True)
    A, B, y, _ = xent_inputs(800 + T, T, K, V)
    w = torch.full((T,), dloss, device="cuda")
    w[: T // 2 : 2] = 0                      # rows that a mask leaves out
    lse = ref.xent(A, B, y)[1][0].float()
    (wA, oA), (wB, oB) = common_dloss(w, A, B, y, lse)
    for kw in ({}, {"work_bytes": T * 1024 + 64 * T * K}):
        dA, dB = ag.gemm_xent_bwd(w, A, B, y, lse, **kw)
        ref.near(dA, wA, oA, "dA %s" % kw)
        ref.near(dB, wB, oB, "dB %s" % kw)


def test_dloss_of_any_values():
    """Zeros, infinities and NaN where there is no target, values of every scale elsewhere, the first ones too."""
    T, K, V = 200, 264, 1003
    A, B, y, _ = xent_inputs(900, T, K, V)
    lse = ref.xent(A, B, y)[1][0].float()
    g = torch.Generator().manual_seed(901)
    w = (torch.randn(T, generator=g) * 2.0 ** torch.randint(-60, 60, (T,), generator=g)).cuda()
    for first in (0.0, 1e-30, 3e38, float("inf"), float("nan"), -2.0):
        v, t = w.clone(), y.clone()
        v[:150], t[:150] = first, -100
        print("dloss", first, flush=True)
        dA, dB = ag.gemm_xent_bwd(v, A, B, t, lse)
        (wA, oA), (wB, oB) = ref.xent_bwd(torch.where(t >= 0, v, torch.zeros_like(v)), A, B, t, lse)
        ref.near(dA, wA, oA, "dA")
        ref.near(dB, wB, oB, "dB")
        assert not dA[:150].any()
