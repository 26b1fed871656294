"""newton_schulz where a factor far from one stands before X or a step: norms far below eps, small coefficients, none before
X itself."""
import pytest
import torch

import allgather_gemm_amd as ag
from ortho_reference import bound, exact, off, spectrum

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


# the kernels of up to 128 and 256 rows, 64 x 64 tiles, those in parts, 128 x 128 tiles, 192 x 192 and 256 x 256 ones
SHAPES = [(64, 100), (200, 320), (320, 200), (500, 1003), (640, 7000), (2050, 2048), (4096, 4224)]


@pytest.mark.parametrize("shape", SHAPES)
def test_norms_far_below_eps(shape):
    """X = G / (|G| + eps) is then about G / eps, and so small that fp16 of X itself has no bits left of it."""
    G = torch.randn(*shape, generator=gen(sum(shape)))
    G /= torch.linalg.vector_norm(G)
    s, n = spectrum(G)
    large = min(shape) > 2000
    for i, (norm, eps) in enumerate([(1e-15, 1e-7), (1e-3, 1.0), (1e-6, 1.0), (1e-9, 1.0), (1e-20, 1.0)][:2 if large else 5]):
        H = (G * norm).to((BF16, torch.float32)[i % 2]).cuda()
        got = ag.newton_schulz(H, eps=eps)
        o, most = off(got, exact(H, ag.NEWTON_SCHULZ, eps)), bound(s * norm, n, ag.NEWTON_SCHULZ, H.dtype == torch.float32, eps)
        print("newton_schulz", shape, norm, eps, "%.2e of %.2e" % (o, most), flush=True)
        assert o <= most, (shape, norm, eps, o, most)


@pytest.mark.parametrize("shape", SHAPES[:4])
def test_largest_eps(shape):
    """A norm of 1 beside eps of 3e38, in steps that bring the result back into bf16's range, and steps enough to bring any back."""
    G = torch.randn(*shape, generator=gen(sum(shape) + 3))
    G = (G / torch.linalg.vector_norm(G)).cuda()
    s, n = spectrum(G)
    for steps in (ag.NEWTON_SCHULZ * 2, ag.NEWTON_SCHULZ * 4):
        o, most = off(ag.newton_schulz(G, coefficients=steps, eps=3e38), exact(G, steps, 3e38)), bound(s, n, steps, True, 3e38)
        print("newton_schulz", shape, len(steps), "%.2e of %.2e" % (o, most), flush=True)
        assert o <= most, (shape, len(steps), o, most)
    assert bool(torch.isfinite(ag.newton_schulz(G, coefficients=ag.NEWTON_SCHULZ * 30, eps=3e38)).all())


def test_stack_of_all_norms():
    """Each matrix of a stack as it is alone, whatever the others' norms; zeros stay zeros."""
    g = gen(1)
    G = torch.randn(6, 300, 520, generator=g)
    for e, norm in enumerate((1.0, 1e-15, 0.0, 1e-7, 1e-30, 1e10)):
        G[e] *= norm / 395
    G = G.cuda()
    out = ag.newton_schulz(G)
    s, n = spectrum(G[0] / torch.linalg.vector_norm(G[0].double()))
    for e in range(6):
        assert torch.equal(out[e], ag.newton_schulz(G[e].contiguous())), e
        norm = float(torch.linalg.vector_norm(G[e].double()))
        if norm == 0:
            assert bool((out[e] == 0).all())
        else:
            assert off(out[e], exact(G[e], ag.NEWTON_SCHULZ)) <= bound(s * norm, n, ag.NEWTON_SCHULZ, True), e


def test_eps_without_a_matrix():
    """Zeros over any eps."""
    for eps in (1e-38, 1e-7, 1.0, 3e38):
        assert bool((ag.newton_schulz(torch.zeros(5, 70, device="cuda"), eps=eps) == 0).all()), eps


@pytest.mark.parametrize("shape", SHAPES[:5])
def test_small_last_steps(shape):
    """A last step that makes X small: out = B X with a B that fp16 of a fixed scale would not hold."""
    G = torch.randn(*shape, generator=gen(sum(shape) + 1)).cuda()
    s, n = spectrum(G)
    for a in (1e-6, 1e-9, 1e-11, 1e-20, 1e-30):
        for steps in ([(a, 0.0, 0.0)], [(a, -a, 0.3 * a)], [(2.0, -1.5, 0.5)] * 2 + [(-a, a, 0.0)]):
            o, most = off(ag.newton_schulz(G, coefficients=steps), exact(G, steps)), bound(s, n, steps, True)
            print("newton_schulz", shape, steps[-1], "%.2e of %.2e" % (o, most), flush=True)
            assert o <= most, (shape, steps[-1], o, most)


@pytest.mark.parametrize("shape", SHAPES[:4])
def test_steps_without_a(shape):
    """Steps in which X is hardly scaled, as far as they are taken: B is next to nothing but A."""
    G = torch.randn(*shape, generator=gen(sum(shape) + 2)).cuda()
    s, n = spectrum(G)
    for steps in ([(0.0, 1.0, 0.0)], [(0.0, 0.0, 1.0)], [(1e-4, 1.0, 0.0)] * 2, [(0.0, 2.0, 0.0), (1.5, -0.5, 0.0)],
                  [(0.0, 1.0, 0.0)] * 2)[:5 if len(s) <= 256 else 4]:
        o, most = off(ag.newton_schulz(G, coefficients=steps), exact(G, steps)), bound(s, n, steps, True)
        print("newton_schulz", shape, steps, "%.2e of %.2e" % (o, most), flush=True)
        assert o <= most, (shape, steps, o, most)
