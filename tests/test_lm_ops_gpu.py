"""gemm_bias_act, gemm_grouped, gemm_xent and their gradients on the GPU against float64, element by element
within the bound that their roundings allow (lm_reference.py)."""
import itertools

import pytest
import torch

import allgather_gemm_amd as ag
import lm_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(BF16).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def guarded(rows, cols):
    """A (rows, cols) bf16 view with sentinels right before and after it, and a check of them."""
    n, pad = rows * cols, 64
    buf = torch.full((n + 2 * pad,), 7.5, dtype=BF16, device="cuda")
    view = buf[pad:pad + n].view(rows, cols)
    view.fill_(float("nan"))
    return view, lambda: bool((buf[:pad] == 7.5).all()) and bool((buf[pad + n:] == 7.5).all())


ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
# one row to many, one column to many, odd sizes around each tile, reductions of less than a step, long ones
# over few tiles, none at all
LINEAR = [(1, 8, 1), (1, 4096, 4096), (2, 64, 7), (3, 0, 9), (16, 2048, 130), (17, 72, 129), (31, 520, 255), (33, 64, 128),
          (48, 1024, 3001), (64, 8192, 40), (65, 320, 384), (129, 200, 257), (256, 128, 128), (300, 1000, 1003),
          (513, 4096, 520), (2100, 256, 2304), (2049, 136, 2311), (60, 6992, 97), (17, 6992, 97), (33, 4000, 1503)]


@pytest.mark.parametrize("i,shape", list(enumerate(LINEAR)))
def test_linear_forward(i, shape):
    M, K, Nc = shape
    g = gen(100 + i)
    A, B = normal(g, M, K), normal(g, Nc, K, std=max(K, 1) ** -0.5)
    for act, with_bias, with_res in itertools.islice(itertools.cycle(itertools.product(ACTS, (True, False), (False, True))),
                                                     i, i + 4 * 5, 4):
        print("linear", shape, act, with_bias, with_res, flush=True)
        bias = normal(g, Nc) if with_bias else None
        res = normal(g, M, Nc) if with_res else None
        C, ok_c = guarded(M, Nc)
        pre, ok_p = guarded(M, Nc)
        out = ag.gemm_bias_act(A, B, bias=bias, act=act, residual=res, C=C, pre=pre)
        assert out.data_ptr() == C.data_ptr()
        y, y_off, p, p_off = ref.linear(A, B, bias, act, res)
        ref.near(C, y, y_off, "C")
        ref.near(pre, p, p_off, "pre")
        assert ok_c() and ok_p()


# enough output for a round of tiles and more (those that the plans send to the tallest ones: test_lm_kernels_gpu.py)
LARGE = [(4100, 72, 4360), (2200, 136, 8200), (5000, 64, 6001), (4353, 200, 4090), (300, 64, 33000)]


@pytest.mark.parametrize("i,shape", list(enumerate(LARGE)))
def test_linear_forward_and_backward_large(i, shape):
    M, K, Nc = shape
    g = gen(150 + i)
    A, B = normal(g, M, K), normal(g, Nc, K, std=max(K, 1) ** -0.5)
    for act, with_bias, with_res in (("none", False, False), (ACTS[1 + i % 4], True, i % 2 == 0)):
        print("linear large", shape, act, flush=True)
        bias = normal(g, Nc) if with_bias else None
        res = normal(g, M, Nc) if with_res else None
        C, ok_c = guarded(M, Nc)
        pre, ok_p = guarded(M, Nc)
        ag.gemm_bias_act(A, B, bias=bias, act=act, residual=res, C=C, pre=pre if with_bias else None)
        y, y_off, p, p_off = ref.linear(A, B, bias, act, res)
        ref.near(C, y, y_off, "C")
        if with_bias:
            ref.near(pre, p, p_off, "pre")
        assert ok_c() and ok_p()
    # the products of the backward pass with M, K and Nc in turn as their large output
    for m, k, n in ((M, Nc // 8 * 8, K), (K, Nc // 8 * 8, M)):
        print("linear bwd large", m, k, n, flush=True)
        A, B, dC = normal(g, m, k), normal(g, n, k, std=0.1), normal(g, m, n)
        got = ag.gemm_bias_act_bwd(dC, A, B)
        for name, t, (want, off) in zip(("dA", "dB", "dbias"), got, ref.linear_bwd(dC, A, B, "none", None)):
            ref.near(t, want, off, name)


def test_linear_residual_in_place():
    g = gen(3)
    A, B, C = normal(g, 70, 256), normal(g, 200, 256, std=0.06), normal(g, 70, 200)
    y, off, _, _ = ref.linear(A, B, None, "silu", C.clone())
    ag.gemm_bias_act(A, B, act="silu", residual=C, C=C)
    ref.near(C, y, off, "C")


LINEAR_BWD = [(1, 8, 1), (1, 1024, 2048), (7, 64, 33), (0, 64, 40), (5, 0, 24), (9, 64, 0), (32, 512, 1000), (33, 136, 129),
              (250, 264, 515), (600, 128, 4104), (2048, 2304, 136), (2100, 264, 2305), (4100, 72, 200)]


@pytest.mark.parametrize("i,shape", list(enumerate(LINEAR_BWD)))
def test_linear_backward(i, shape):
    M, K, Nc = shape
    g = gen(200 + i)
    A, B, dC, pre = normal(g, M, K), normal(g, Nc, K, std=0.1), normal(g, M, Nc), normal(g, M, Nc, std=1.5)
    for act in ACTS:
        print("linear bwd", shape, act, flush=True)
        got = ag.gemm_bias_act_bwd(dC, A, B, act=act, pre=None if act == "none" else pre)
        for name, t, (want, off) in zip(("dA", "dB", "dbias"), got, ref.linear_bwd(dC, A, B, act, pre)):
            assert t.shape == want.shape
            ref.near(t, want, off, "%s %s" % (act, name))
    only = ag.gemm_bias_act_bwd(dC, A, B, act="relu", pre=pre, need_dA=False, need_dbias=False)
    assert only[0] is None and only[2] is None
    ref.near(only[1], *ref.linear_bwd(dC, A, B, "relu", pre)[1], "dB alone")


def test_linear_activation_slope_at_zero_and_far_out():
    pre = torch.tensor([[0.0, -0.0, 60.0, -60.0, 3e38, -3e38, 1e-38, -20.0]], dtype=BF16, device="cuda")
    dC = torch.ones_like(pre)
    A, B = torch.ones(1, 8, dtype=BF16, device="cuda"), torch.zeros(8, 8, dtype=BF16, device="cuda")
    for act in ACTS[1:]:
        got = ag.gemm_bias_act_bwd(dC, A, B, act=act, pre=pre)[2].double()
        want = {"relu": [0, 0, 1, 0, 1, 0, 1, 0]}.get(act, [0.5, 0.5, 1, 0, 1, 0, 0.5, 0])
        assert torch.allclose(got.cpu(), torch.tensor(want, dtype=torch.float64), atol=1e-6), (act, got)


def test_offsets_past_32_bits():
    """Outputs and weights of more than 2^32 bytes: the last rows and the last expert."""
    g = gen(17)
    M, K, Nc = 70000, 16, 32776
    A, B, bias = normal(g, M, K), normal(g, Nc, K), normal(g, Nc)
    print("linear", M, K, Nc, flush=True)
    C = ag.gemm_bias_act(A, B, bias=bias, act="relu", residual=None)
    for rows in (slice(0, 200), slice(65400, 65700), slice(M - 200, M)):
        y, off, _, _ = ref.linear(A[rows], B, bias, "relu", None)
        ref.near(C[rows], y, off, "C")
    print("linear dA", flush=True)
    dA = ag.gemm_bias_act_bwd(C, A, B, need_dB=False, need_dbias=False)[0]
    ref.near(dA[-100:], *ref.linear_bwd(C[-100:], A[-100:], B, "none", None)[0], "dA")
    del C, dA
    E, K, Nc = 9, 16384, 16384
    W = torch.zeros(E, Nc, K, dtype=BF16, device="cuda")
    W[-1] = normal(g, Nc, 8).repeat(1, K // 8)
    A, dC = normal(g, 40, K), normal(g, 40, Nc)
    ends = torch.tensor([0, 10, 10, 10, 10, 10, 10, 10, 40], dtype=torch.int32, device="cuda")
    print("grouped", E, K, Nc, flush=True)
    got = ag.gemm_grouped(A, W, ends)
    want, off = ref.product(A[10:].double(), W[-1].double())
    ref.near(got[10:], want, off * (1 + ref.H) + ref.H * want.abs(), "grouped C")
    assert not got[:10].any()
    dW = ag.gemm_grouped_bwd(dC, A, W, ends, need_dA=False)[1]
    want, off = ref.product(dC[10:].double().t().contiguous(), A[10:].double().t().contiguous())
    ref.near(dW[-1], want, off * (1 + ref.H) + ref.H * want.abs(), "grouped dB")
    assert not dW[0].any() and dW[1].any() and not dW[2:8].any()


def ends_of(sizes):
    return torch.tensor(list(itertools.accumulate(sizes)), dtype=torch.int32, device="cuda")


# sizes of the groups, rows that belong to none, K, Nc
GROUPED = [([1], 0, 8, 8), ([0, 0, 3], 2, 64, 40), ([5, 0, 1, 0, 0, 9, 2], 0, 72, 136), ([0, 0], 4, 64, 64),
           ([2] * 16, 0, 2048, 512), ([33, 1, 0, 200, 31], 7, 136, 264), ([130, 127, 128, 129], 1, 520, 384),
           ([700, 0, 5, 300, 256], 90, 264, 520), ([64, 0, 3, 100] * 80, 11, 64, 72), ([1] * 1024, 3, 64, 16),
           ([900, 257, 256, 255], 0, 0, 48)]
# groups that end inside a tile, many rows; weights large enough for the tallest tiles of dB
GROUPED += [([700, 513, 0, 1200, 130, 2, 128, 384, 640, 1], 33, 136, 2056), ([257] * 12, 0, 72, 1544),
            ([300, 0, 1, 511, 64, 900, 256], 5, 2056, 1288)]


@pytest.mark.parametrize("i,case", list(enumerate(GROUPED)))
def test_grouped_forward_and_backward(i, case):
    sizes, spare, K, Nc = case
    M, E = sum(sizes) + spare, len(sizes)
    print("grouped", E, M, K, Nc, flush=True)
    g = gen(300 + i)
    A, B, dC = normal(g, M, K), normal(g, E, Nc, K, std=0.1), normal(g, M, Nc)
    ends = ends_of(sizes)
    C, ok = guarded(M, Nc)
    ag.gemm_grouped(A, B, ends, C=C)
    ref.near(C, *ref.grouped(A, B, ends.tolist()), "C")
    assert ok() and not C[sum(sizes):].any()
    dA, dB = ag.gemm_grouped_bwd(dC, A, B, ends)
    (wA, oA), (wB, oB) = ref.grouped_bwd(dC, A, B, ends.tolist())
    ref.near(dA, wA, oA, "dA")
    ref.near(dB, wB, oB, "dB")
    assert not dA[sum(sizes):].any()
    for e, n in enumerate(sizes):
        assert n or not dB[e].any()
    a, b = ag.gemm_grouped_bwd(dC, A, B, ends, need_dB=False)
    assert b is None and torch.equal(a, dA)


def test_grouped_rows_of_none_hold_nothing_of_what_is_there():
    """Infinities and NaN in rows past the last group, and in the weights of groups without rows, reach nothing."""
    g = gen(5)
    A, B, dC = normal(g, 40, 64), normal(g, 4, 48, 64), normal(g, 40, 48)
    ends = ends_of([10, 0, 20, 0])
    clean = [t.clone() for t in (ag.gemm_grouped(A, B, ends), *ag.gemm_grouped_bwd(dC, A, B, ends))]
    A[30:], dC[30:], B[1], B[3] = float("nan"), float("inf"), float("nan"), float("inf")
    dirty = [ag.gemm_grouped(A, B, ends), *ag.gemm_grouped_bwd(dC, A, B, ends)]
    for x, y in zip(clean, dirty):
        assert torch.equal(x, y)


@pytest.mark.parametrize("table", [[10, 5, 30], [-7, 0, 90], [50, 40, 30], [2 ** 31 - 1, -(2 ** 31), 0]])
def test_grouped_tables_that_are_no_running_sums_stay_in_bounds(table):
    g = gen(6)
    M, K, Nc = 40, 64, 48
    A, B, dC = normal(g, M, K), normal(g, 3, Nc, K, std=0.1), normal(g, M, Nc)
    ends = torch.tensor(table, dtype=torch.int32, device="cuda")
    C, ok = guarded(M, Nc)
    ag.gemm_grouped(A, B, ends, C=C)
    ref.near(C, *ref.grouped(A, B, table), "C")
    assert ok()
    (wA, oA), (wB, oB) = ref.grouped_bwd(dC, A, B, table)
    dA, dB = ag.gemm_grouped_bwd(dC, A, B, ends)
    ref.near(dA, wA, oA, "dA")
    ref.near(dB, wB, oB, "dB")


XENT = [(1, 8, 1), (1, 1024, 5000), (3, 64, 2), (8, 256, 1003), (33, 128, 999), (100, 520, 2049), (130, 64, 300),
        (257, 136, 1025), (300, 0, 17), (700, 264, 4099), (107, 3176, 1003), (65, 1280, 4427), (1024, 640, 515)]


@pytest.mark.parametrize("i,shape", list(enumerate(XENT)))
def test_xent_forward_and_backward(i, shape):
    T, K, V = shape
    print("xent", shape, flush=True)
    g = gen(400 + i)
    A, B = normal(g, T, K), normal(g, V, K, std=2 * max(K, 1) ** -0.5)
    y = torch.randint(0, V, (T,), generator=g).cuda()
    y[0], y[-1] = V - 1, 0
    if T > 2:
        y[1] = -100
    if T > 30:
        y[20], y[21], y[22] = V, -1, 2 ** 62
    loss, lse = ag.gemm_xent(A, B, y)
    (wl, ol), (ws, os_), _, _ = ref.xent(A, B, y)
    ref.near(loss, wl, ol, "loss")
    ref.near(lse, ws, os_, "lse")
    dloss = torch.rand(T, generator=g).cuda() * 2 - 0.5
    dA, dB = ag.gemm_xent_bwd(dloss, A, B, y, lse)
    (wA, oA), (wB, oB) = ref.xent_bwd(dloss, A, B, y, lse)
    ref.near(dA, wA, oA, "dA")
    ref.near(dB, wB, oB, "dB")
    if T > 2:
        assert loss[1] == 0 and not dA[1].any()
    # a vocabulary in many pieces: the same gradients
    small = 1 << 20
    if T <= 300:
        pA, pB = ag.gemm_xent_bwd(dloss, A, B, y, lse, work_bytes=small)
        ref.near(pA, wA, oA, "dA in pieces")
        ref.near(pB, wB, oB, "dB in pieces")
        assert ag.gemm_xent_bwd(dloss, A, B, y, lse, need_dA=False)[0] is None


def test_xent_in_many_pieces():
    g = gen(7)
    T, K, V = 300, 264, 3001
    A, B = normal(g, T, K), normal(g, V, K, std=0.1)
    y = torch.randint(0, V, (T,), generator=g).cuda()
    loss, lse = ag.gemm_xent(A, B, y)
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    (wA, oA), (wB, oB) = ref.xent_bwd(dloss, A, B, y, lse)
    # each of the twelve pieces adds its own fp32 sum: covered by the bound's count of products
    for n in (900 << 10, 1200 << 10):
        dA, dB = ag.gemm_xent_bwd(dloss, A, B, y, lse, work_bytes=n)
        ref.near(dA, wA, oA, "dA")
        ref.near(dB, wB, oB, "dB")


def test_xent_no_rows():
    A, B = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(50, 64, dtype=BF16, device="cuda")
    y, f = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = ag.gemm_xent(A, B, y)
    dA, dB = ag.gemm_xent_bwd(f, A, B, y, lse)
    assert loss.numel() == lse.numel() == dA.numel() == 0 and not dB.any()


def test_xent_large_and_infinite_logits():
    """Logits of thousands leave the statistics finite; a logit of minus infinity has no weight; a row whose
    logits hold NaN or plus infinity has a NaN loss and leaves the other rows as they are."""
    K, V = 64, 700
    A = torch.zeros(4, K, dtype=BF16, device="cuda")
    B = torch.zeros(V, K, dtype=BF16, device="cuda")
    A[:, 0] = torch.tensor([100.0, 1.0, -1.0, 0.5]).to(BF16)
    B[:, 0] = torch.linspace(-90, 90, V).to(BF16)
    A[1, 1] = 1.0
    B[5, 1] = float("-inf")            # 0 * inf in rows 0, 2, 3 is NaN; row 1 gets -inf
    y = torch.tensor([3, 7, 9, 11], device="cuda")
    loss, lse = ag.gemm_xent(A, B, y)
    z = A.double() @ B.double().t()
    want = torch.logsumexp(z[1], 0)
    assert torch.isnan(loss[[0, 2, 3]]).all()
    assert abs(float(lse[1]) - float(want)) < 1e-4 and abs(float(loss[1]) - float(want - z[1, 7])) < 1e-4
    B[5, 1] = 0
    loss, lse = ag.gemm_xent(A, B, y)
    (wl, ol), (ws, os_), _, _ = ref.xent(A, B, y)
    ref.near(loss, wl, ol, "loss")
    ref.near(lse, ws, os_, "lse")


def test_gradients_against_differences():
    """<gradient, direction> against the central difference of the float64 forward form along it."""
    g = gen(9)
    M, K, Nc, V = 40, 64, 72, 333
    h = 1e-4

    def direction(shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64).cuda()

    def check(f, x, grad, off, what):
        d = direction(x.shape)
        slope = (f(x.double() + h * d) - f(x.double() - h * d)) / (2 * h)
        got = (grad.double() * d).sum()
        # the gradient's own bound along the direction, and h^2 times a third derivative of order one per element
        assert abs(float(got - slope)) <= float((off * d.abs()).sum()) + 1e-5 * float(d.abs().sum()), what

    A, B, bias, dC = normal(g, M, K), normal(g, Nc, K, std=0.1), normal(g, Nc), normal(g, M, Nc)
    for act in ("silu", "gelu", "gelu_tanh"):
        pre = torch.empty(M, Nc, dtype=BF16, device="cuda")
        ag.gemm_bias_act(A, B, bias=bias, act=act, pre=pre)
        got = ag.gemm_bias_act_bwd(dC, A, B, act=act, pre=pre)
        bounds = ref.linear_bwd(dC, A, B, act, pre)
        # pre is stored in bf16: its half step times the slope's own slope (at most 1.2) is in d
        extra = 1.2 * ref.H * pre.double().abs() * dC.double().abs()

        def f(a, b, c):
            return (dC.double() * ref.act_value(a @ b.t() + c, act)).sum()
        a64, b64, c64 = A.double(), B.double(), bias.double()
        check(lambda x: f(x, b64, c64), A, got[0], bounds[0][1] + extra @ b64.abs(), act + " dA")
        check(lambda x: f(a64, x, c64), B, got[1], bounds[1][1] + extra.t() @ a64.abs(), act + " dB")
        check(lambda x: f(a64, b64, x), bias, got[2], bounds[2][1] + extra.sum(0), act + " dbias")
    ends = ends_of([11, 0, 20, 5])
    W = normal(g, 4, Nc, K, std=0.1)
    dA, dW = ag.gemm_grouped_bwd(dC, A, W, ends)
    (_, oA), (_, oW) = ref.grouped_bwd(dC, A, W, ends.tolist())

    def fg(a, w):
        return sum((dC[lo:hi].double() * (a[lo:hi] @ w[e].t())).sum() for e, (lo, hi) in enumerate(ref.spans(ends.tolist(), M)))
    check(lambda x: fg(x, W.double()), A, dA, oA, "grouped dA")
    check(lambda x: fg(A.double(), x), W, dW, oW, "grouped dB")
    Bv = normal(g, V, K, std=0.2)
    y = torch.randint(0, V, (M,), generator=g).cuda()
    y[4] = -100
    loss, lse = ag.gemm_xent(A, Bv, y)
    w = torch.rand(M, generator=g).cuda()
    dA, dB = ag.gemm_xent_bwd(w, A, Bv, y, lse)
    (_, oA), (_, oB) = ref.xent_bwd(w, A, Bv, y, lse)

    def fx(a, b):
        z = a @ b.t()
        rows = torch.nonzero(y >= 0).flatten()
        return (w.double()[rows] * (torch.logsumexp(z, 1)[rows] - z[rows, y[rows]])).sum()
    check(lambda x: fx(x, Bv.double()), A, dA, oA, "xent dA")
    check(lambda x: fx(A.double(), x), Bv, dB, oB, "xent dB")


def test_same_inputs_same_bits_and_other_streams():
    """No result depends on the order of workgroups, nor on the stream."""
    g = gen(11)
    A, B, W = normal(g, 200, 1024), normal(g, 264, 1024, std=0.05), normal(g, 5, 264, 1024, std=0.05)
    dC, pre = normal(g, 200, 264), normal(g, 200, 264)
    ends = ends_of([50, 0, 100, 7, 40])
    y = torch.randint(0, 264, (200,), generator=g).cuda()
    w = torch.rand(200, generator=g).cuda()

    def everything(stream=None):
        loss, lse = ag.gemm_xent(A, B, y, stream=stream)
        return [ag.gemm_bias_act(A, B, act="silu", stream=stream), *ag.gemm_bias_act_bwd(dC, A, B, "gelu", pre, stream=stream),
                ag.gemm_grouped(A, W, ends, stream=stream), *ag.gemm_grouped_bwd(dC, A, W, ends, stream=stream),
                loss, lse, *ag.gemm_xent_bwd(w, A, B, y, lse, stream=stream)]
    first = everything()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for out in (everything(), everything(side)):
        torch.cuda.synchronize()
        for p, q in zip(first, out):
            assert torch.equal(p, q)


def test_calls_replay_from_a_graph():
    """A training step's calls captured once, replayed over changed inputs, each replay against the eager result."""
    g = gen(13)
    A, B, V = normal(g, 96, 512), normal(g, 200, 512, std=0.05), normal(g, 1000, 200, std=0.1)
    y = torch.randint(0, 1000, (96,), generator=g).cuda()
    w = torch.full((96,), 1 / 96, device="cuda")

    def step():
        pre = torch.empty(96, 200, dtype=BF16, device="cuda")
        h = ag.gemm_bias_act(A, B, act="gelu", pre=pre)
        loss, lse = ag.gemm_xent(h, V, y)
        dh, dV = ag.gemm_xent_bwd(w, h, V, y, lse)
        dA, dB, db = ag.gemm_bias_act_bwd(dh, A, B, act="gelu", pre=pre)
        return loss, dV, dA, dB, db
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        A.copy_(normal(gen(50 + i), 96, 512))
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, step()):
            assert torch.equal(p, q), i
