"""newton_schulz's error against the bound that follows from its roundings, spectrum by spectrum (ortho_reference.py), for the default
coefficients and for others that are in use, those that start at a = 8.2 among them."""
import pytest
import torch

import allgather_gemm_amd as ag
from ortho_reference import bound, exact, off, spectrum

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

STEPS = {
    "default": ag.NEWTON_SCHULZ,
    "default, twice": ag.NEWTON_SCHULZ * 2,
    "cubic": [(1.5, -0.5, 0.0)] * 12,
    "quintic": [(2.0, -1.5, 0.5)] * 8,
    "large, then fine": list(ag.NEWTON_SCHULZ[:3]) + [(2.0, -1.5, 0.5)] * 3,
    # steps fitted one after the other, of a falling from 8.2 on
    "fitted": [(8.2052, -22.9019, 16.4607), (4.0664, -2.8612, 0.5184), (3.9096, -2.8234, 0.525),
               (3.2856, -2.4153, 0.4853), (2.2779, -1.6198, 0.3985)],
}


def spectra():
    g = torch.Generator().manual_seed(17)
    m, n = 512, 700
    Q = [torch.linalg.qr(torch.randn(k, m, generator=g, dtype=torch.float64))[0] for k in (m, n)]
    yield "powers", (Q[0] * torch.arange(1, m + 1) ** -1.5) @ Q[1].t()
    yield "six decades", (Q[0] * torch.logspace(0, -6, m)) @ Q[1].t()
    yield "few gradients", (torch.randn(m, 32, generator=g) * torch.rand(1, 32, generator=g) ** 4) @ torch.randn(32, n, generator=g)
    yield "shared directions", (torch.randn(m, 64, generator=g) / torch.arange(1, 65)) @ torch.randn(64, n, generator=g) + \
        0.05 * torch.randn(m, n, generator=g)
    yield "rows of many scales", torch.randn(m, n, generator=g) * torch.exp(3 * torch.randn(m, 1, generator=g))
    yield "random", torch.randn(m, n, generator=g)
    yield "orthogonal", Q[0] @ Q[1].t()
    yield "random, 64 rows", torch.randn(64, 100, generator=g)
    yield "random, long", torch.randn(100, 5440, generator=g)
    yield "random, 1100 rows", torch.randn(1100, 1300, generator=g)


@pytest.mark.parametrize("name,G", list(spectra()), ids=lambda v: v if isinstance(v, str) else "")
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_error_within_the_roundings(name, G, dtype):
    G = G.to(dtype)
    s, n = spectrum(G)
    G = G.cuda()
    T = G.t().contiguous()
    for what, steps in STEPS.items():
        most, want = bound(s, n, steps, dtype == torch.float32), exact(G, steps)
        for H, w in ((G, want), (T, want.t())):
            o = off(ag.newton_schulz(H, coefficients=steps), w)
            print("%s, %s: %.2e of %.2e" % (name, what, o, most), flush=True)
            assert o <= most, (name, what, o, most)
