"""Plain float64 forms of the language-model operators, with an elementwise bound of the error that the
kernels' stated roundings allow.

Half a step of bf16 is H = 2^-8 relative, of fp32 F = 2^-24.  An fp32 sum of n products in any order is off
by at most (n + 8) F times the sum of their magnitudes (products of two bf16 are exact in fp32; the matrix
instructions' internal order and the joining of splits are covered by n; 8 covers what follows the sum).
exp(x) by exp2 of the rounded x log2(e) is off by about (|x| + 4) F relative; E = 2^-18 covers it, and the
reciprocal and erf next to it, for the |x| <= 40 where the result is not negligible.
"""
import math

import torch

H, F, E = 2.0 ** -8, 2.0 ** -24, 2.0 ** -18


def act_value(x, act):
    if act == "relu":
        return torch.relu(x)          # slope 0 at 0
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * 0.5 * torch.special.erfc(-x / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    return x


def act_slope(x, act):
    x = x.detach().clone().requires_grad_(True)
    with torch.enable_grad():
        y = act_value(x, act).sum()
        return torch.autograd.grad(y, x)[0] if act != "none" else torch.ones_like(x)


def product(a, b):
    """(a b^T, its error bound) for 2D float64 a (m, k), b (n, k)."""
    return a @ b.t(), (a.shape[1] + 8) * F * (a.abs() @ b.abs().t())


def linear(A, B, bias, act, residual):
    """(C, its bound, pre, its bound).  No activation's slope exceeds 1.13."""
    pre, off = product(A.double(), B.double())
    if bias is not None:
        pre = pre + bias.double()
        off = off + F * pre.abs() * 2
    y = act_value(pre, act)
    y_off = 1.13 * off + (E * (y.abs() + pre.abs()) if act not in ("none", "relu") else 0)
    if residual is not None:
        y = y + residual.double()
        y_off = y_off + 2 * F * y.abs()
    return y, y_off * (1 + H) + H * y.abs(), pre, off * (1 + H) + H * pre.abs()


def linear_bwd(dC, A, B, act, pre):
    """((dA, bound), (dB, bound), (dbias, bound)): d is rounded to bf16 before the products."""
    d = dC.double()
    d_off = torch.zeros_like(d)
    if act != "none":
        d = d * act_slope(pre.double(), act)
        d_off = E * (d.abs() + dC.double().abs()) if act != "relu" else d_off
    dr_off = d_off * (1 + H) + (H * d.abs() if act != "none" else 0)
    a, b = A.double(), B.double()
    dA, offA = product(d, b.t().contiguous())
    dB, offB = product(d.t().contiguous(), a.t().contiguous())
    offA = offA * (1 + H) + dr_off @ b.abs()
    offB = offB * (1 + H) + dr_off.t() @ a.abs()
    dbias = d.sum(0)
    off = d_off.sum(0) + (d.shape[0] + 8) * F * d.abs().sum(0)
    return ((dA, offA * (1 + H) + H * dA.abs()), (dB, offB * (1 + H) + H * dB.abs()),
            (dbias, off * (1 + H) + H * dbias.abs()))


def spans(ends, M):
    """Row ranges of the groups, a table's entries held to the range that their predecessors leave."""
    out, prev = [], 0
    for e in ends:
        e = max(prev, min(int(e), M))
        out.append((prev, e))
        prev = e
    return out


def grouped(A, B, ends):
    a, b = A.double(), B.double()
    C = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64, device=a.device)
    off = torch.zeros_like(C)
    for e, (lo, hi) in enumerate(spans(ends, a.shape[0])):
        C[lo:hi], off[lo:hi] = product(a[lo:hi], b[e])
    return C, off * (1 + H) + H * C.abs()


def grouped_bwd(dC, A, B, ends):
    d, a, b = dC.double(), A.double(), B.double()
    dA, offA = torch.zeros_like(a), torch.zeros_like(a)
    dB, offB = torch.zeros_like(b), torch.zeros_like(b)
    for e, (lo, hi) in enumerate(spans(ends, a.shape[0])):
        dA[lo:hi], offA[lo:hi] = product(d[lo:hi], b[e].t().contiguous())
        dB[e], offB[e] = product(d[lo:hi].t().contiguous(), a[lo:hi].t().contiguous())
    return (dA, offA * (1 + H) + H * dA.abs()), (dB, offB * (1 + H) + H * dB.abs())


def xent(A, B, targets):
    """((loss, bound), (lse, bound), logits, their bound)."""
    z, off = product(A.double(), B.double())
    lse = torch.logsumexp(z, 1)
    lse_off = off.amax(1) + E + 4 * F * lse.abs()
    has = (targets >= 0) & (targets < B.shape[0])
    hit = torch.where(has, targets, 0).unsqueeze(1)
    loss = torch.where(has, lse - z.gather(1, hit).squeeze(1), 0.0)
    loss_off = torch.where(has, lse_off + off.gather(1, hit).squeeze(1) + F * loss.abs(), 0.0)
    return (loss, loss_off), (lse, lse_off), z, off


def xent_bwd(dloss, A, B, targets, lse):
    """((dA, bound), (dB, bound)) with the given fp32 lse taken as it is."""
    a, b, g = A.double(), B.double(), dloss.double()
    z, off = product(a, b)
    has = (targets >= 0) & (targets < B.shape[0])
    w = torch.where(has, g, 0.0).unsqueeze(1)
    p = torch.exp(z - lse.double().unsqueeze(1))
    p_off = p * (torch.expm1(off + F * lse.double().abs().unsqueeze(1)) + E)
    hit = torch.where(has, targets, 0).unsqueeze(1)
    D = (p - torch.zeros_like(p).scatter_(1, hit, 1.0)) * w
    D_off = (p_off + 4 * F) * w.abs() * (1 + H) + H * D.abs()
    dA, offA = product(D, b.t().contiguous())
    dB, offB = product(D.t().contiguous(), a.t().contiguous())
    offA = offA * (1 + H) + D_off @ b.abs()
    offB = offB * (1 + H) + D_off.t() @ a.abs()
    return (dA, offA * (1 + H) + H * dA.abs()), (dB, offB * (1 + H) + H * dB.abs())


def near(got, want, bound, what=""):
    """Every element inside its bound (plus the smallest normal's scale, for results that round to zero)."""
    d = (got.double() - want).abs()
    ok = (d <= bound + 1e-30) | ~torch.isfinite(want)
    assert bool(ok.all()), "%s: %d of %d outside, worst %.3g times its bound" % (
        what, int((~ok).sum()), ok.numel(), float((d / (bound + 1e-30))[torch.isfinite(want)].max()))
    assert bool(torch.isfinite(got[torch.isfinite(want)]).all()), what
