"""layer_norm and layer_norm_bwd on the GPU against float64, element by element within the bound that their roundings allow.

An fp32 sum that a value reaches through at most D additions is off by at most D F times the sum of the magnitudes.  No value
of a row passes more than width / 1024 + 100 of them (its thread's, six steps between lanes, one for each wave); a
column's at most one for each row and 8 + 100 where partial sums are joined."""
import itertools

import pytest
import torch

import allgather_gemm_amd as ag
from lm_reference import F, H, near

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS = 1e-5


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=g) * std + mean).to(BF16).cuda()


def guarded(rows, cols, dtype=BF16):
    n, pad = rows * cols, 64
    buf = torch.full((n + 2 * pad,), 7.5, dtype=dtype, device="cuda")
    view = buf[pad:pad + n].view(rows, cols)
    view.fill_(float("nan"))
    return view, lambda: bool((buf[:pad] == 7.5).all()) and bool((buf[pad + n:] == 7.5).all())


def depth(width):
    return width / 1024 + 100


def forward(s, w, b, eps):
    """((y, bound), (mean, bound), (rstd, bound)) for the normalised rows s."""
    D = depth(s.shape[1])
    s = s.double()
    mean = s.mean(1, keepdim=True)
    mean_off = (D + 2) * F * s.abs().mean(1, keepdim=True)
    d = s - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    rel = ((D + 4) * F * var + mean_off ** 2) / (var + eps) / 2 + 4 * F
    w = torch.ones_like(s[0]) if w is None else w.double()
    b = torch.zeros_like(s[0]) if b is None else b.double()
    xh = d * rstd
    y = xh * w + b
    off = w.abs() * rstd * (mean_off + 2 * F * d.abs()) * (1 + rel) + (xh * w).abs() * rel + 4 * F * ((xh * w).abs() + b.abs())
    return (y, off * (1 + H) + H * y.abs()), (mean[:, 0], mean_off[:, 0]), (rstd[:, 0], (rstd * rel)[:, 0])


def backward(dy, h, mean, rstd, w, dh):
    """((dx, bound), (dw, bound), (db, bound)), the fp32 statistics taken as they are."""
    D, T = depth(h.shape[1]), h.shape[0]
    dy, mean, rstd = dy.double(), mean.double().unsqueeze(1), rstd.double().unsqueeze(1)
    xh = (h.double() - mean) * rstd
    g = dy if w is None else dy * w.double()
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    o1, o2 = (D + 3) * F * g.abs().mean(1, keepdim=True), (D + 6) * F * (g * xh).abs().mean(1, keepdim=True)
    dx = rstd * (g - m1 - xh * m2)
    off = rstd * (o1 + xh.abs() * o2 + 8 * F * (g.abs() + m1.abs() + (xh * m2).abs()))
    if dh is not None:
        dx = dx + dh.double()
        off = off + F * dh.double().abs()
    dw, db = (dy * xh).sum(0), dy.sum(0)
    dwo, dbo = (T + 112) * F * (dy * xh).abs().sum(0), (T + 108) * F * dy.abs().sum(0)
    return tuple((v, o * (1 + H) + H * v.abs()) for v, o in ((dx, off + 2 * F * dx.abs()), (dw, dwo), (db, dbo)))


# every number of threads and pieces that a row's width asks for, its borders, odd widths, one column, the widest in registers
# and beyond
WIDTHS = [1, 2, 7, 8, 9, 64, 127, 128, 129, 256, 257, 500, 512, 513, 1003, 1024, 1025, 2047, 2048, 2049, 4095, 4096, 4097,
          8191, 8192, 8193, 14336, 16383, 16384, 16385, 20001, 40008]
ROWS = [1, 2, 3, 5, 17, 33, 128, 256, 257]


@pytest.mark.parametrize("i,width", list(enumerate(WIDTHS)))
def test_forward_and_backward(i, width):
    g = gen(300 + i)
    kinds = itertools.cycle([(True, True, True), (False, True, False), (True, False, True), (False, False, False)])
    for rows, (add, with_w, with_b) in zip((ROWS[i % 9], ROWS[(i * 4 + 3) % 9], 1), kinds):
        print("norm", rows, width, add, with_w, with_b, flush=True)
        x = (torch.randn(rows, width, generator=g) * torch.randn(width, generator=g).exp() + torch.randn(rows, 1, generator=g)).to(BF16).cuda()
        res = normal(g, rows, width, std=3.0) if add else None
        w = normal(g, width, std=0.3, mean=1.0) if with_w else None
        b = normal(g, width) if with_b else None
        s = (x.float() + res.float()).to(BF16) if add else x
        y, ok_y = guarded(rows, width)
        h, ok_h = guarded(rows, width)
        mean, ok_m = guarded(1, rows, torch.float32)
        rstd, ok_r = guarded(1, rows, torch.float32)
        out = ag.layer_norm(x, weight=w, bias=b, eps=EPS, residual=res, y=y, h=h if add else None, mean=mean[0], rstd=rstd[0])
        assert out.data_ptr() == y.data_ptr()
        for name, got, (want, off) in zip(("y", "mean", "rstd"), (y, mean[0], rstd[0]), forward(s, w, b, EPS)):
            near(got, want, off, name)
        if add:
            assert torch.equal(h, s)
        assert ok_y() and ok_h() and ok_m() and ok_r()
        # without what only the backward pass needs: the same bits
        assert torch.equal(ag.layer_norm(x, weight=w, bias=b, eps=EPS, residual=res), y)
        dy = normal(g, rows, width)
        dh = normal(g, rows, width) if i % 3 else None
        got = ag.layer_norm_bwd(dy, s, mean[0], rstd[0], weight=w, dh=dh)
        for name, t, (want, off) in zip(("dx", "dw", "db"), got, backward(dy, s, mean[0], rstd[0], w, dh)):
            near(t, want, off, name)
        only = ag.layer_norm_bwd(dy, s, mean[0], rstd[0], weight=w, dh=dh, need_dweight=False, need_dbias=False)
        assert only[1] is None and only[2] is None and torch.equal(only[0], got[0])
        only = ag.layer_norm_bwd(dy, s, mean[0], rstd[0], weight=w, dh=dh, need_dx=False, need_dbias=False)
        assert only[0] is None and only[2] is None and torch.equal(only[1], got[1])


# more rows than a launch has workgroups for, and enough for many partial sums
MANY = [(20001, 72), (9000, 200), (5003, 500), (5003, 1000), (5000, 1504), (4100, 4096), (2100, 6000), (1500, 9001), (700, 17000)]


@pytest.mark.parametrize("rows,width", MANY)
def test_many_rows(rows, width):
    g = gen(rows)
    print("norm", rows, width, flush=True)
    x, res, w, b, dy, dh = (normal(g, *s) for s in ((rows, width), (rows, width), (width,), (width,), (rows, width), (rows, width)))
    h = torch.empty_like(x)
    mean, rstd = torch.empty(2, rows, device="cuda")
    y = ag.layer_norm(x, weight=w, bias=b, eps=EPS, residual=res, h=h, mean=mean, rstd=rstd)
    s = (x.float() + res.float()).to(BF16)
    assert torch.equal(h, s)
    for name, got, (want, off) in zip(("y", "mean", "rstd"), (y, mean, rstd), forward(s, w, b, EPS)):
        near(got, want, off, name)
    for more in (None, dh):
        first = ag.layer_norm_bwd(dy, h, mean, rstd, weight=w, dh=more)
        for name, t, (want, off) in zip(("dx", "dw", "db"), first, backward(dy, h, mean, rstd, w, more)):
            near(t, want, off, name)
    # the sums' order is the shape's alone
    for t, u in zip(first, ag.layer_norm_bwd(dy, h, mean, rstd, weight=w, dh=dh)):
        assert torch.equal(t, u)


def test_no_rows_and_no_columns():
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    stat = torch.empty(0, device="cuda")
    assert ag.layer_norm(x, mean=stat, rstd=stat).shape == (0, 64)
    dx, dw, db = ag.layer_norm_bwd(x, x, stat, stat)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())
    x = torch.empty(5, 0, dtype=BF16, device="cuda")
    stat = torch.zeros(5, device="cuda")
    assert ag.layer_norm(x).shape == (5, 0)
    assert [t.numel() for t in ag.layer_norm_bwd(x, x, stat, stat)] == [0, 0, 0]


@pytest.mark.parametrize("width", [9, 1000, 4096, 20000])
def test_rows_that_do_not_vary_and_far_offsets(width):
    """A constant row is its bias; a row far from zero keeps its variance (the differences from the mean are summed, not squares)."""
    b = torch.linspace(-2, 2, width).to(BF16).cuda()
    x = torch.full((2, width), 3.0, dtype=BF16, device="cuda")
    x[1] = 0
    assert torch.equal(ag.layer_norm(x, bias=b), b.expand(2, width))
    g = gen(7)
    x = (1024 + 8 * torch.randint(-3, 4, (4, width), generator=g).float()).to(BF16).cuda()
    mean, rstd = torch.empty(2, 4, device="cuda")
    y = ag.layer_norm(x, eps=EPS, mean=mean, rstd=rstd)
    for name, got, (want, off) in zip(("y", "mean", "rstd"), (y, mean, rstd), forward(x, None, None, EPS)):
        near(got, want, off, name)
    # the squares' mean less the mean's square would be off by 2^-24 1024^2 = 0.06 of a variance of about 256
    v = x.double().var(1, correction=0)
    assert float(((rstd.double() ** -2 - EPS) / v - 1).abs().max()) < 2e-5


@pytest.mark.parametrize("width", [500, 4097, 17000])
def test_rows_with_nan_and_infinity_stay_apart(width):
    g = gen(8)
    x, dy = normal(g, 6, width), normal(g, 6, width)
    clean = ag.layer_norm(x)
    x[1, width - 1], x[4, 0] = float("nan"), float("inf")
    mean, rstd = torch.empty(2, 6, device="cuda")
    y = ag.layer_norm(x, mean=mean, rstd=rstd)
    for row in range(6):
        assert bool(torch.isnan(y[row]).all()) if row in (1, 4) else torch.equal(y[row], clean[row])
    dx = ag.layer_norm_bwd(dy, x, mean, rstd, need_dweight=False, need_dbias=False)[0]
    assert bool(torch.isfinite(dx[[0, 2, 3, 5]]).all()) and bool(torch.isnan(dx[[1, 4]]).all())


@pytest.mark.parametrize("width", [1003, 4096, 20000])
def test_sum_in_place(width):
    g = gen(9)
    x, res, w = normal(g, 37, width), normal(g, 37, width), normal(g, width)
    want_h = (x.float() + res.float()).to(BF16)
    want = ag.layer_norm(want_h, weight=w)
    r = res.clone()
    assert torch.equal(ag.layer_norm(x, weight=w, residual=r, h=r), want) and torch.equal(r, want_h)
    r = x.clone()
    assert torch.equal(ag.layer_norm(r, weight=w, residual=res, h=r), want) and torch.equal(r, want_h)


def test_gradients_by_differences():
    """The gradients against differences of the formula in float64, in a direction of each input."""
    g = gen(10)
    rows, width = 9, 264
    x, w, b, dy, dh = normal(g, rows, width), normal(g, width), normal(g, width), normal(g, rows, width), normal(g, rows, width)
    mean, rstd = torch.empty(2, rows, device="cuda")
    ag.layer_norm(x, weight=w, bias=b, eps=EPS, mean=mean, rstd=rstd)
    got = ag.layer_norm_bwd(dy, x, mean, rstd, weight=w, dh=dh)

    def value(x, w, b):
        d = x - x.mean(1, keepdim=True)
        y = d * ((d * d).mean(1, keepdim=True) + EPS) ** -0.5 * w + b
        return (y * dy.double()).sum() + (x * dh.double()).sum()
    at = [t.double() for t in (x, w, b)]
    for i in range(3):
        v = torch.randn(at[i].shape, generator=g, dtype=torch.float64).cuda()
        plus, minus = list(at), list(at)
        plus[i], minus[i] = at[i] + 1e-4 * v, at[i] - 1e-4 * v
        slope = float(value(*plus) - value(*minus)) / 2e-4
        # each of the gradient's values is rounded by at most H of it; 1e-5: the differences' own error
        off = float((got[i].double() * v).abs().sum()) * H * 1.1 + 1e-5 * abs(slope) + 1e-4
        assert abs(float((got[i].double() * v).sum()) - slope) <= off, i


def test_graph_and_streams():
    g = gen(11)
    rows, width = 700, 2056
    x, res, w, b, dy = normal(g, rows, width), normal(g, rows, width), normal(g, width), normal(g, width), normal(g, rows, width)
    h = torch.empty_like(x)
    mean, rstd = torch.empty(2, rows, device="cuda")

    def step():
        y = ag.layer_norm(x, weight=w, bias=b, residual=res, h=h, mean=mean, rstd=rstd)
        return (y,) + ag.layer_norm_bwd(dy, h, mean, rstd, weight=w, dh=y)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ag.layer_norm(x, weight=w, bias=b, residual=res, stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    for i in range(4):
        x.copy_(normal(g, rows, width))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, u in zip(out, step()):
            assert torch.equal(t, u), i


@pytest.mark.parametrize("width", [9, 100, 1003, 4097, 20001])
def test_mean_times_rstd_past_fp32(width):
    """A constant row's gradient is finite though its mean times its rstd is not: nothing past the row's end takes part."""
    g = gen(13)
    x = torch.full((300, width), 2.0 ** 110, dtype=BF16, device="cuda")
    w, dy = normal(g, width), normal(g, 300, width)
    mean, rstd = torch.empty(2, 300, device="cuda")
    ag.layer_norm(x, eps=1e-12, mean=mean, rstd=rstd)
    assert bool((mean == 2.0 ** 110).all()) and bool(torch.isinf(mean * rstd).all())
    for rows in (300, 2):
        got = ag.layer_norm_bwd(dy[:rows], x[:rows], mean[:rows], rstd[:rows], weight=w)
        for name, t, (want, off) in zip(("dx", "dw", "db"), got, backward(dy[:rows], x[:rows], mean[:rows], rstd[:rows], w, None)):
            near(t, want, off, name)


# more than 2^32 values, for every way through memory
@pytest.mark.parametrize("rows,width", [(45000000, 100), (1100000, 4096), (260000, 17000)])
def test_offsets_past_32_bits(rows, width):
    print("norm", rows, width, flush=True)
    g = gen(14)
    n = 300
    x = torch.zeros(rows, width, dtype=BF16, device="cuda")
    dy = torch.zeros_like(x)
    x[-n:], dy[-n:] = normal(g, n, width), normal(g, n, width)
    mean, rstd = torch.empty(2, rows, device="cuda")
    y = ag.layer_norm(x, eps=EPS, mean=mean, rstd=rstd)
    at = [t[-n:] for t in (y, mean, rstd)]
    for name, got, (want, off) in zip(("y", "mean", "rstd"), at, forward(x[-n:], None, None, EPS)):
        near(got, want, off, name)
    assert bool((y[:n] == 0).all()) and bool((y[-2 * n:-n] == 0).all())
    del y
    dx, dw, db = ag.layer_norm_bwd(dy, x, mean, rstd)
    for name, t, (want, off) in zip(("dx", "dw", "db"), (dx[-n:], dw, db), backward(dy[-n:], x[-n:], at[1], at[2], None, None)):
        near(t, want, off, name)
    assert bool((dx[:n] == 0).all()) and bool((dx[-2 * n:-n] == 0).all())


def test_two_streams_at_once():
    g = gen(15)
    sets = []
    for rows, width in ((5000, 1504), (256, 4096)):
        x, res, w, dy = normal(g, rows, width), normal(g, rows, width), normal(g, width), normal(g, rows, width)

        def step(x=x, res=res, w=w, dy=dy):
            h = torch.empty_like(x)
            mean, rstd = torch.empty(2, x.shape[0], device="cuda")
            y = ag.layer_norm(x, weight=w, residual=res, h=h, mean=mean, rstd=rstd)
            return (y, h) + ag.layer_norm_bwd(dy, h, mean, rstd, weight=w)
        sets.append((step, step(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(5):
        got = []
        for step, want, stream in sets:
            with torch.cuda.stream(stream):
                got.append([step() for _ in range(3)])
        torch.cuda.synchronize()
        for (step, want, stream), outs in zip(sets, got):
            for out in outs:
                assert all(torch.equal(t, u) for t, u in zip(out, want)), i


@pytest.mark.parametrize("rows,width", [(33, 1003), (256, 4096), (700, 203), (700, 1003), (600, 4097), (520, 9001), (300, 20001), (9, 7)])
def test_gradient_added_in_place(rows, width):
    """The C entry point with dx in dh's buffer, every kernel that has a dh, odd row ends."""
    g = gen(16)
    h, w, dy, dh = normal(g, rows, width), normal(g, width), normal(g, rows, width), normal(g, rows, width)
    mean, rstd = torch.empty(2, rows, device="cuda")
    ag.layer_norm(h, eps=EPS, mean=mean, rstd=rstd)
    want = ag.layer_norm_bwd(dy, h, mean, rstd, weight=w, dh=dh)
    got = dh, torch.empty_like(w), torch.empty_like(w)
    n = ag.lib().layer_norm_bwd_workspace(rows, width)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    rc = ag.lib().layer_norm_bwd(*(t.data_ptr() for t in (dy, h, mean, rstd, w, dh)), rows, width, *(t.data_ptr() for t in got),
                                 work.data_ptr() if n else None, n, torch.cuda.current_stream().cuda_stream)
    assert rc == ag.AG_OK
    assert all(torch.equal(t, u) for t, u in zip(got, want))
