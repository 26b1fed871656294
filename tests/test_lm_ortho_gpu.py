"""newton_schulz on the GPU against float64.

Every matrix that a step stores (X, A, B = b A + c A A) is rounded to fp16, half a step of which is 2^-11 of a value, and the
result to bf16, 2^-8.  Spread evenly over its step, a rounding is off by 1 / sqrt(3) of that in the root of the mean square.
To first order a step turns an error e of X into a e + ..., at most max |p'| <= a of it among small singular directions, where
the kept remainder leaves none, and about one elsewhere; X's rounding reaches a step's result through B (|B| <= 2.81 for the
default coefficients), A's as (b + 2 c t) s, at most 4.8, B's as s, at most 1.2.  Independent of each other, five steps'
are sqrt(5 (2.81^2 + 4.8^2 + 1.2^2)) 2^-11 / sqrt(3) = 3.6e-3, and with the result's 2.26e-3 4.3e-3 of the result's norm.
All of one sign and at their largest, for matrices too small for an average: 2^-8 + 5 (2.81 + 4.8 + 1.2) 2^-11 = 2.6e-2."""
import pytest
import torch

import allgather_gemm_amd as ag

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
OFF, OFF_SMALL = 4.3e-3, 2.6e-2
EPS = 1e-7


def gen(seed):
    return torch.Generator().manual_seed(seed)


def exact(G, steps=ag.NEWTON_SCHULZ, eps=EPS):
    X = G.double()
    if X.shape[0] > X.shape[1]:
        return exact(G.t().contiguous(), steps, eps).t()
    X = X / (torch.linalg.vector_norm(X) + eps)
    for a, b, c in steps:
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X


def off(got, want):
    assert bool(torch.isfinite(got).all())
    return float(torch.linalg.vector_norm(got.double() - want) / torch.linalg.vector_norm(want))


def near(G, got, steps=ag.NEWTON_SCHULZ, what="", eps=EPS):
    assert got.dtype == BF16 and got.shape == G.shape
    most = OFF if min(G.shape) >= 16 else OFF_SMALL
    o = off(got, exact(G, steps, eps))
    print(what, tuple(G.shape), "%.2e" % o, flush=True)
    assert o <= most, (what, tuple(G.shape), o)


# one element to many, a row, a column, odd extents, borders of the padding and of both tiles, tall and wide
SHAPES = [(1, 1), (1, 9), (9, 1), (2, 3), (7, 300), (300, 7), (16, 16), (64, 64), (65, 127), (128, 128), (129, 128), (128, 129),
          (130, 257), (256, 256), (257, 255), (500, 1003), (1003, 500), (512, 256), (640, 1000), (1000, 1000), (1280, 4100), (4100, 1280),
          (100, 5440), (8000, 250), (640, 8192), (1030, 1100), (1024, 2048), (1500, 1600)]


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_shapes(i, shape, dtype):
    print("newton_schulz", shape, dtype, flush=True)
    G = (torch.randn(*shape, generator=gen(i)) * 10.0 ** (i % 7 - 3)).to(dtype).cuda()
    n, pad = G.numel(), 64
    buf = torch.full((n + 2 * pad,), 7.5, dtype=BF16, device="cuda")
    out = buf[pad:pad + n].view(shape)
    before = G.clone()
    got = ag.newton_schulz(G, out=out)
    assert got.data_ptr() == out.data_ptr() and torch.equal(G, before)
    near(G, got)
    assert bool((buf[:pad] == 7.5).all()) and bool((buf[pad + n:] == 7.5).all())
    assert torch.equal(ag.newton_schulz(G), got)


# a round of the large tiles and more, for all three products, odd numbers of them
LARGE = [(2050, 2048), (4096, 4224), (4000, 5000), (6016, 6016), (9000, 2100)]


@pytest.mark.parametrize("shape", LARGE)
def test_large(shape):
    print("newton_schulz", shape, flush=True)
    G = torch.randn(*shape, generator=gen(shape[0])).cuda()
    near(G, ag.newton_schulz(G))


def spectra():
    g = gen(3)
    m, n = 512, 700
    Q = [torch.linalg.qr(torch.randn(k, m, generator=g, dtype=torch.float64))[0] for k in (m, n)]
    yield "powers", (Q[0] * torch.arange(1, m + 1) ** -1.5) @ Q[1].t()
    yield "six decades", (Q[0] * torch.logspace(0, -6, m)) @ Q[1].t()
    yield "few gradients", (torch.randn(m, 32, generator=g) * torch.rand(1, 32, generator=g) ** 4) @ torch.randn(32, n, generator=g)
    yield "shared directions", (torch.randn(m, 64, generator=g) / torch.arange(1, 65)) @ torch.randn(64, n, generator=g) + \
        0.05 * torch.randn(m, n, generator=g)
    yield "rows of many scales", torch.randn(m, n, generator=g) * torch.exp(3 * torch.randn(m, 1, generator=g))
    yield "one direction", torch.outer(torch.randn(m, generator=g), torch.randn(n, generator=g))
    yield "orthogonal", Q[0] @ Q[1].t()


@pytest.mark.parametrize("name,G", list(spectra()), ids=lambda v: v if isinstance(v, str) else "")
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_spectra(name, G, dtype):
    """Small singular values among large ones: their directions keep what one fp16 would lose (to 2e-2)."""
    G = G.to(dtype).cuda()
    for H in (G, G.t().contiguous()):
        near(H, ag.newton_schulz(H), what=name)


def test_sizes_of_values():
    """The norm is taken out exactly: the largest and smallest magnitudes, and a power of two changes nothing."""
    g = gen(4)
    G = torch.randn(200, 320, generator=g).cuda()
    want = ag.newton_schulz(G, eps=0.0)
    for k in (-100, -60, 60, 110):
        assert torch.equal(ag.newton_schulz(G * 2.0 ** k, eps=0.0), want), k
    for scale in (3e-38, 1e-30, 1e30, 5e37):
        H = G * scale
        near(H, ag.newton_schulz(H, eps=0.0), what=str(scale), eps=0.0)
        H = H.to(BF16)
        near(H, ag.newton_schulz(H, eps=0.0), what=str(scale), eps=0.0)
    # eps next to a small norm: what is left of it
    H = (G * 1e-9).float()
    assert off(ag.newton_schulz(H, eps=1e-6), exact(H, eps=float(torch.tensor(1e-6)))) <= OFF


def test_zeros_infinities_and_nan():
    G = torch.zeros(3, 100, 140, device="cuda")
    G[1] = torch.randn(100, 140, generator=gen(5)).cuda()
    out = ag.newton_schulz(G)
    assert bool((out[0] == 0).all()) and bool((out[2] == 0).all())
    assert torch.equal(out[1], ag.newton_schulz(G[1].contiguous()))
    for bad in (float("nan"), float("inf"), float("-inf")):
        G[2, 7, 9] = bad
        out = ag.newton_schulz(G)
        assert bool(torch.isnan(out[2]).all()) and bool((out[0] == 0).all()) and bool(torch.isfinite(out[1]).all())
    assert bool(torch.isnan(ag.newton_schulz(torch.zeros(4, 5, device="cuda"), eps=0.0)).all())
    assert ag.newton_schulz(torch.zeros(0, 5, 6, device="cuda")).shape == (0, 5, 6)
    assert ag.newton_schulz(torch.zeros(5, 0, device="cuda")).shape == (5, 0)


STACKS = [(2, 64, 100), (5, 300, 130), (7, 129, 513), (16, 1024, 600), (40, 72, 72), (3, 2100, 2050), (3, 200, 4000), (2, 640, 7000),
          (4, 1100, 1024), (16, 520, 1000)]


@pytest.mark.parametrize("E,R,C", STACKS)
def test_stacks(E, R, C):
    print("stack", E, R, C, flush=True)
    g = gen(E)
    G = torch.randn(E, R, C, generator=g).to(BF16)
    G[E // 2] *= 1e-3
    G = G.cuda()
    out = ag.newton_schulz(G)
    for e in range(E):
        near(G[e], out[e])
    # in place
    H = G.clone()
    assert ag.newton_schulz(H, out=H) is H and torch.equal(H, out)


def test_other_coefficients():
    g = gen(6)
    G = torch.randn(160, 300, generator=g).cuda()
    for steps in ([(1.5, -0.5, 0.0)] * 3, [(1.0, 0.0, 0.0)], [(0.0, 0.0, 0.0)], [(1.875, -1.25, 0.375)] * 7,
                  [(2.0, -1.5, 0.5), (3.4445, -4.7750, 2.0315)], [(-1.0, 0.25, 0.0)] * 2):
        got, want = ag.newton_schulz(G, coefficients=steps), exact(G, steps)
        if float(want.abs().max()) == 0:
            assert bool((got == 0).all())
        else:
            assert off(got, want) <= OFF, steps
    with pytest.raises(ag.AgError, match=r"\(-5\)"):
        ag.newton_schulz(G, coefficients=[(10.0, 0.0, 0.0)] * 2)
    with pytest.raises(ag.AgError, match=r"\(-1\)"):
        ag.newton_schulz(G, coefficients=[(float("nan"), 0.0, 0.0)])


def test_graph_and_streams():
    g = gen(12)
    G = torch.randn(3, 400, 264, generator=g).cuda()
    want = ag.newton_schulz(G)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ag.newton_schulz(G, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        ag.newton_schulz(G)
        with torch.cuda.graph(graph, stream=side):
            out = ag.newton_schulz(G)
    for i in range(4):
        G.copy_(torch.randn(3, 400, 264, generator=g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ag.newton_schulz(G)), i


def test_offsets_past_32_bits():
    """A stack of more than 2^32 elements, its first and last matrix the only ones that are not zeros."""
    E, n = 140, 5600
    print("stack", E, n, n, flush=True)
    G = torch.zeros(E, n, n, dtype=BF16, device="cuda")
    for e in (0, E - 1):
        G[e] = torch.randn(n, n, generator=gen(20 + e)).to(BF16).cuda()
    out = ag.newton_schulz(G)
    for e in (0, E - 1):
        near(G[e], out[e])
    assert bool((out[1] == 0).all()) and bool((out[E - 2] == 0).all())


def test_two_streams_at_once():
    """Products in parts, whose counts live in each call's own workspace, and large ones beside them."""
    sets = []
    for i, shape in enumerate(((640, 8192), (100, 5440), (1100, 1024))):
        G = torch.randn(*shape, generator=gen(30 + i)).cuda()
        sets.append((G, ag.newton_schulz(G), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(5):
        got = []
        for G, want, stream in sets:
            got.append([ag.newton_schulz(G, stream=stream) for _ in range(3)])
        torch.cuda.synchronize()
        for (G, want, stream), outs in zip(sets, got):
            assert all(torch.equal(out, want) for out in outs), (i, tuple(G.shape))


@pytest.mark.parametrize("shape", [(640, 8192), (250, 8000), (72, 72)])
def test_parts_in_a_graph(shape):
    g = gen(13)
    G = torch.randn(*shape, generator=g).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        ag.newton_schulz(G)
        with torch.cuda.graph(graph, stream=side):
            out = ag.newton_schulz(G)
    for i in range(4):
        G.copy_(torch.randn(*shape, generator=g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ag.newton_schulz(G)), i
