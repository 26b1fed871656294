"""newton_schulz in float64, and how far the roundings that lm_ortho.hip states may take a result from it.

X, A and B = a I + b A + c A A are stored as fp16, half a step of which is 2^-11 of a value; the result as bf16, 2^-8.  A rounding
spread over its step has a root of the mean square of at most U = 2^-11 / sqrt(3) of a value, and one whose entries are
independent of each other looks the same in every orthogonal basis: in the basis of X's singular vectors an error's entries
all have the mean square ||error||^2 / entries.  There a step's derivative is known: of an error's symmetric and
antisymmetric part it makes d1 = (p_i - p_j) / (s_i - s_j) and d2 = (p_i + p_j) / (s_i + s_j) times that, and p / s of what lies
outside the square, for X's singular values s and p = a s + b s^3 + c s^5.  What a step adds itself, to first order:

  X's rounding without a remainder     goes through the step as X does: times d1, d2, p / s
  ... with one                         A and B X take the value alone, a X is whole: times d1 - a, d2 - a, p / s - a
  A's, entries e of U ||A||            (b + c (t_i + t_j)) e s_j, t = s^2
  B's beside the diagonal              e s_j, entries of U ||b A + c A A||
  B's diagonal                         entries that are nearly equal round alike: all of 2^-11 and one sign, X times 1 + 2^-11,
                                       which later steps multiply by s p' / p; these add up, the others' squares do

A remainder is kept behind a step while the product of the a's to come is above 8, and before the first one for an fp32 G; a bf16
G starts without rounding.  The result's own rounding joins at the end.  15 % on top cover that a norm over a few thousand
roundings is not its mean, the terms of second order and the fp32 sums (sqrt(n) 2^-24).
"""
import math

import torch

U = 2.0 ** -11 / math.sqrt(3)
EPS = 1e-7


def exact(G, steps, eps=EPS):
    X = G.double()
    if X.shape[0] > X.shape[1]:
        return exact(G.t().contiguous(), steps, eps).t()
    X = X / (torch.linalg.vector_norm(X) + float(torch.tensor(eps, dtype=torch.float32)))
    for a, b, c in steps:
        A = X @ X.t()
        X = a * X + (b * A + c * (A @ A)) @ X
    return X


def spectrum(G):
    """Singular values (of the smaller extent's number) and the larger extent, on the CPU."""
    X = G.double()
    X = X.t() if X.shape[0] > X.shape[1] else X
    return torch.linalg.eigvalsh((X @ X.t()).cpu()).clamp(min=0).sqrt(), X.shape[1]


def bound(s, n, steps, fp32, eps=EPS):
    """Most that the result's error may be of the result's norm, for G's singular values s and larger extent n."""
    s = s / (torch.linalg.vector_norm(s) + eps)
    s = s.clamp(min=float(s.max()) * 1e-9)
    m = len(s)
    sym, anti, out, bias = torch.zeros(m, m, dtype=s.dtype), torch.zeros(m, m, dtype=s.dtype), torch.zeros(m, dtype=s.dtype), torch.zeros_like(s)

    def kept(i):
        return math.prod(abs(q[0]) for q in steps[i + 1:]) > 8
    for i, (a, b, c) in enumerate(steps):
        t = s * s
        p, slope = s * (a + b * t + c * t * t), a + 3 * b * t + 5 * c * t * t
        near = (s[:, None] - s[None]).abs() <= 1e-6 * s[:, None]
        d1 = torch.where(near, slope[:, None].expand(m, m), (p[:, None] - p[None]) / torch.where(near, 1.0, s[:, None] - s[None]))
        d2 = (p[:, None] + p[None]) / (s[:, None] + s[None])
        whole = kept(i - 1) and (i > 0 or fp32)            # X's remainder is there
        x = 0.0 if i == 0 and not fp32 else U * U * float(t.sum()) / (m * n)     # mean square of X's rounding
        off = a if whole else 0.0
        sym = sym * d1 ** 2 + x / 2 * (d1 - off) ** 2
        anti = anti * d2 ** 2 + x / 2 * (d2 - off) ** 2
        out = out * (p / s) ** 2 + (n - m) * x * (p / s - off) ** 2
        for k, square in ((b + c * (t[:, None] + t[None]), float((t * t).sum())), (1.0, float(((b * t + c * t * t) ** 2).sum()))):
            e = U * U * square / (m * m) * k * k
            sym = sym + e * (s[:, None] + s[None]) ** 2 / 4
            anti = anti + e * (s[:, None] - s[None]) ** 2 / 4
        bias = bias * slope.abs() + 2.0 ** -11 * s * (a + b * t + c * t * t).abs()
        s = p.abs().clamp(min=float(p.abs().max()) * 1e-12)
    square = float(sym.sum() + anti.sum() + out.sum() + (bias ** 2).sum())
    return 1.15 * math.sqrt(square / float((s * s).sum()) + 2.0 ** -16 / 3)


def off(got, want):
    assert bool(torch.isfinite(got).all())
    return float(torch.linalg.vector_norm(got.double() - want) / torch.linalg.vector_norm(want))
