"""Calls that between them launch every kernel of the language-model operators, and with the tallest tiles every way
that those are cut: whole, in pairs of groups' halves, in halves and in quarters.  test_lm_launches.py holds the shapes
below and those of test_lm_ops_gpu.py to that.  Against float64, within the bounds of lm_reference.py."""
import itertools

import pytest
import torch

import allgather_gemm_amd as ag
import lm_reference as ref
from test_lm_ops_gpu import ACTS, BF16, ends_of, gen, guarded, normal

pytestmark = pytest.mark.gpu

# M, K, Nc, activation, bias, residual, pre: the tallest tiles with what may follow the sums, and alone; few rows over
# many columns
LINEAR = [(6041, 1320, 1228, "gelu", True, True, True), (8992, 824, 1570, "relu", True, False, True),
          (7198, 688, 2740, "gelu_tanh", False, True, False), (6381, 832, 2750, "silu", True, True, True),
          (5325, 744, 1482, "none", False, False, False), (1660, 1920, 2712, "none", False, False, False),
          (4353, 1000, 4090, "none", True, True, False),
          (1, 32768, 97, "silu", True, True, True), (9, 8200, 1001, "gelu", True, False, True),
          (40, 16392, 4601, "relu", False, True, False),
          (52, 200, 70, "gelu", True, True, True), (36, 264, 4750, "silu", True, True, True),
          (51, 136, 4923, "relu", False, True, True), (11, 328, 5003, "gelu", True, False, False),
          (19, 200, 4266, "gelu_tanh", True, True, True), (23, 136, 4700, "none", False, True, False)]
# M, K, Nc, activation: gradients' tallest tiles, and dA's reduction split over them
LINEAR_BWD = [(2632, 2880, 591, "gelu_tanh"), (3247, 1184, 8574, "gelu"), (687, 2936, 2597, "silu"), (4353, 1000, 4090, "none"),
              (61, 72, 50, "relu")]
# groups' rows, rows of none, the long side of the output and the reduction: the first in quarters, the second in halves
TALL_GROUPS = [([306, 514, 0, 74, 174, 0, 80, 903, 1410, 133, 26, 1347], 77, 2936),
               ([416, 649, 741, 40, 406, 371, 760, 201, 706, 406, 9, 566], 77, 3224)]
GROUPED_FWD = [(sizes, spare, k, wide) for sizes, spare, wide in TALL_GROUPS for k in (72, 392)]
GROUPED_BWD = [(sizes, spare, wide, k) for sizes, spare, wide in TALL_GROUPS for k in (72, 392)]
# few rows a group: sizes, rows of none, K, Nc
GROUPED_FEW = [([4, 0, 9], 2, 264, 1624), ([4, 3], 0, 200, 2504), ([49, 65, 13, 0, 24], 0, 136, 392), ([34, 0], 3, 72, 40),
               ([0, 64, 20, 15], 20, 136, 2056), ([3, 0, 1, 17, 0] * 30, 9, 1208, 72), ([2, 0, 5, 0] * 25, 4, 1032, 40),
               ([9, 0, 2] * 70, 3, 512, 136), ([1, 0, 2, 60, 0, 0, 9, 3], 1, 328, 1032)]
# T, K, V
XENT = [(2100, 72, 3001), (4100, 8, 500), (6041, 1320, 1228), (2169, 1544, 3247), (4454, 472, 4109), (3983, 536, 3793), (7198, 688, 2740), (2600, 1000, 6001),
        (16000, 136, 60), (2000, 200, 501), (200, 328, 8000), (1000, 1032, 1500), (19, 264, 4266), (17, 136, 200), (56, 200, 333), (5, 264, 9001), (27, 520, 4611), (36, 264, 4750), (2, 72, 36001)]
# T, K, V, bytes of scratch memory: several pieces of the vocabulary, whose dA are added up by each kernel of dA
XENT_PIECES = [(3247, 1184, 8574, 61594368), (7198, 688, 2740, 24400000), (3, 72, 700, 4096), (20, 200, 3000, 200000),
               (300, 264, 3001, 1 << 20)]


@pytest.mark.parametrize("i,case", list(enumerate(LINEAR)))
def test_linear_forward(i, case):
    M, K, Nc, act, with_bias, with_res, with_pre = case
    print("linear", case, flush=True)
    g = gen(500 + i)
    A, B = normal(g, M, K), normal(g, Nc, K, std=K ** -0.5)
    bias = normal(g, Nc) if with_bias else None
    res = normal(g, M, Nc) if with_res else None
    C, ok_c = guarded(M, Nc)
    pre, ok_p = guarded(M, Nc)
    ag.gemm_bias_act(A, B, bias=bias, act=act, residual=res, C=C, pre=pre if with_pre else None)
    y, y_off, p, p_off = ref.linear(A, B, bias, act, res)
    ref.near(C, y, y_off, "C")
    if with_pre:
        ref.near(pre, p, p_off, "pre")
    assert ok_c() and ok_p()


@pytest.mark.parametrize("i,case", list(enumerate(LINEAR_BWD)))
def test_linear_backward(i, case):
    M, K, Nc, act = case
    print("linear bwd", case, flush=True)
    g = gen(540 + i)
    A, B, dC, pre = normal(g, M, K), normal(g, Nc, K, std=0.1), normal(g, M, Nc), normal(g, M, Nc, std=1.5)
    got = ag.gemm_bias_act_bwd(dC, A, B, act=act, pre=None if act == "none" else pre)
    for name, t, (want, off) in zip(("dA", "dB", "dbias"), got, ref.linear_bwd(dC, A, B, act, pre)):
        ref.near(t, want, off, name)


def grouped_inputs(i, sizes, spare, K, Nc):
    """A, B, dC and ends, with what no result may hold where no group's rows are."""
    M, E = sum(sizes) + spare, len(sizes)
    g = gen(i)
    A, B, dC = normal(g, M, K), normal(g, E, Nc, K, std=0.1), normal(g, M, Nc)
    A[M - spare:], dC[M - spare:] = float("nan"), float("inf")
    clean = B.clone()
    for e, n in enumerate(sizes):
        if n == 0:
            B[e] = float("nan")
    return A, B, dC, ends_of(sizes), clean


@pytest.mark.parametrize("i,case", list(enumerate(GROUPED_FWD + GROUPED_FEW)))
def test_grouped_forward(i, case):
    sizes, spare, K, Nc = case
    print("grouped", sizes, spare, K, Nc, flush=True)
    A, B, _, ends, clean = grouped_inputs(600 + i, *case)
    C, ok = guarded(A.shape[0], Nc)
    ag.gemm_grouped(A, B, ends, C=C)
    ref.near(C, *ref.grouped(A, clean, ends.tolist()), "C")
    assert ok() and not C[sum(sizes):].any()


@pytest.mark.parametrize("i,case", list(enumerate(GROUPED_BWD + GROUPED_FEW)))
def test_grouped_backward(i, case):
    sizes, spare, K, Nc = case
    print("grouped bwd", sizes, spare, K, Nc, flush=True)
    A, B, dC, ends, clean = grouped_inputs(650 + i, *case)
    dA, dB = ag.gemm_grouped_bwd(dC, A, B, ends)
    (wA, oA), (wB, oB) = ref.grouped_bwd(dC, A, clean, ends.tolist())
    ref.near(dA, wA, oA, "dA")
    ref.near(dB, wB, oB, "dB")
    assert not dA[sum(sizes):].any()
    for e, n in enumerate(sizes):
        assert n or not dB[e].any()


def xent_inputs(seed, T, K, V):
    g = gen(seed)
    A, B = normal(g, T, K), normal(g, V, K, std=2 * K ** -0.5)
    y = torch.randint(0, V, (T,), generator=g).cuda()
    y[0], y[-1] = V - 1, 0
    if T > 2:
        y[1] = -100
    if T > 30:
        y[20], y[21], y[22] = V, -1, 2 ** 62
    return A, B, y, torch.rand(T, generator=g).cuda() * 2 - 0.5


@pytest.mark.parametrize("i,case", list(enumerate(XENT)))
def test_xent_forward_and_backward(i, case):
    print("xent", case, flush=True)
    A, B, y, dloss = xent_inputs(700 + i, *case)
    loss, lse = ag.gemm_xent(A, B, y)
    (wl, ol), (ws, os_), _, _ = ref.xent(A, B, y)
    ref.near(loss, wl, ol, "loss")
    ref.near(lse, ws, os_, "lse")
    dA, dB = ag.gemm_xent_bwd(dloss, A, B, y, lse)
    (wA, oA), (wB, oB) = ref.xent_bwd(dloss, A, B, y, lse)
    ref.near(dA, wA, oA, "dA")
    ref.near(dB, wB, oB, "dB")
    none = (y < 0) | (y >= case[2])
    assert not loss[none].any() and not dA[none].any()


@pytest.mark.parametrize("i,case", list(enumerate(XENT_PIECES)))
def test_xent_in_pieces(i, case):
    print("xent in pieces", case, flush=True)
    A, B, y, dloss = xent_inputs(750 + i, *case[:3])
    lse = ref.xent(A, B, y)[1][0].float()
    dA, dB = ag.gemm_xent_bwd(dloss, A, B, y, lse, work_bytes=case[3])
    (wA, oA), (wB, oB) = ref.xent_bwd(dloss, A, B, y, lse)
    ref.near(dA, wA, oA, "dA")
    ref.near(dB, wB, oB, "dB")


def test_every_activation_with_the_tallest_tiles():
    """Bias, residual and pre in turn, into rows that start on no more than two bytes."""
    M, K, Nc = 4353, 1000, 4091
    g = gen(790)
    A, B, bias, res = normal(g, M, K), normal(g, Nc, K, std=K ** -0.5), normal(g, Nc), normal(g, M, Nc)
    for act, (b, r, p) in zip(ACTS, itertools.cycle([(True, True, True), (False, True, False), (True, False, True)])):
        print("linear", (M, K, Nc), act, b, r, p, flush=True)
        C, ok_c = guarded(M, Nc)
        pre = torch.empty(M, Nc, dtype=BF16, device="cuda") if p else None
        ag.gemm_bias_act(A, B, bias=bias if b else None, act=act, residual=res if r else None, C=C, pre=pre)
        y, y_off, q, q_off = ref.linear(A, B, bias if b else None, act, res if r else None)
        ref.near(C, y, y_off, "C")
        if p:
            ref.near(pre, q, q_off, "pre")
        assert ok_c()
