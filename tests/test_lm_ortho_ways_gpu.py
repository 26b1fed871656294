"""newton_schulz on the GPU through every way that its plans choose between (test_ortho_plans.py has that none is left out):
last rounds of tiles in quarters, tiles that share a CU, results that are turned."""
import pytest
import torch

import allgather_gemm_amd as ag
from ortho_reference import bound, exact, off, spectrum

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

# X X^T and A A in 128 x 128 tiles of which the last go in quarters, wide and tall, in stacks; 256 x 256 ones without quarters;
# B X in 256 x 256 tiles with quarters, turned; two 64 x 64 tiles a CU, turned; 128 x 128 ones without quarters, turned
WAYS = [(1, 2880, 2900), (1, 3000, 2870), (16, 2048, 1024), (16, 1000, 2040), (1, 3400, 4000), (64, 396, 393), (1, 4928, 4928),
        (1, 8448, 2112), (16, 2059, 301), (8, 349, 268), (8, 268, 349), (1, 2496, 832)]


@pytest.mark.parametrize("i,stack", list(enumerate(WAYS)), ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else "")
def test_ways(i, stack):
    E, R, C = stack
    G = torch.randn(E, R, C, generator=torch.Generator().manual_seed(100 + i)).to((BF16, torch.float32)[i % 2])
    print("newton_schulz", stack, flush=True)
    s, n = spectrum(G[0])              # the others' are as good as the same
    most = bound(s, n, ag.NEWTON_SCHULZ, i % 2 == 1)
    G = G.cuda()
    count, pad = G.numel(), 64
    buf = torch.full((count + 2 * pad,), 7.5, dtype=BF16, device="cuda")
    out = ag.newton_schulz(G, out=buf[pad:pad + count].view(G.shape))
    for e in range(E):
        o = off(out[e], exact(G[e], ag.NEWTON_SCHULZ))
        if e in (0, E - 1):
            print("newton_schulz", stack, e, "%.2e of %.2e" % (o, most), flush=True)
        assert o <= most, (stack, e, o, most)
    assert bool((buf[:pad] == 7.5).all()) and bool((buf[pad + count:] == 7.5).all())
    assert torch.equal(ag.newton_schulz(G), out)
