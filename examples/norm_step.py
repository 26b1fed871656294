"""A training step of a pre-norm block and head over row shards, its matrices updated by orthogonalised momenta:

    r = gather(shards) W0^T                                    ag_gemm: the residual stream
    h = silu(norm(r) W1^T + b1);  m = h W2^T                   layer_norm, gemm_bias_act
    s = r + m;  loss = cross entropy of norm(s) V^T            layer_norm with the residual in front, gemm_xent

Backwards, layer_norm_bwd adds the gradient that reaches the residual stream beside the norm.  W0, W1 and W2 then move along
newton_schulz of their momentum; the rest goes down its gradient.  Nothing is copied to the host inside a step.

    python examples/norm_step.py          # prints the mean loss of each step
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import allgather_gemm_amd as ag  # noqa: E402
from lm_step import batch  # noqa: E402

BF16 = torch.bfloat16


class Model:
    def __init__(self, width=256, hidden=512, vocab=1003, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).to(BF16)

        def vector(n, value):
            return torch.full((n,), value, dtype=BF16, device="cuda")

        self.W0, self.W1, self.W2, self.V = weight(width, width), weight(hidden, width), weight(width, hidden), weight(vocab, width)
        self.b1 = vector(hidden, 0.0)
        self.g1, self.c1, self.g2, self.c2 = vector(width, 1.0), vector(width, 0.0), vector(width, 1.0), vector(width, 0.0)
        self.momenta = {k: torch.zeros(getattr(self, k).shape, device="cuda") for k in ("W0", "W1", "W2")}

    def parameters(self):
        return {k: getattr(self, k) for k in ("W0", "g1", "c1", "W1", "b1", "W2", "g2", "c2", "V")}

    def forward(self, shards, targets):
        s, rows, width = {}, sum(t.shape[0] for t in shards), self.W0.shape[0]

        def empty(cols):
            return torch.empty(rows, cols, dtype=BF16, device="cuda")
        s["a"], s["pre"], s["s"] = empty(shards[0].shape[1]), empty(self.W1.shape[0]), empty(width)
        s["mean1"], s["rstd1"], s["mean2"], s["rstd2"] = torch.empty(4, rows, device="cuda")
        s["r"] = ag.ag_gemm(shards, self.W0, 128, a_out=s["a"])
        s["y1"] = ag.layer_norm(s["r"], self.g1, self.c1, mean=s["mean1"], rstd=s["rstd1"])
        s["h"] = ag.gemm_bias_act(s["y1"], self.W1, bias=self.b1, act="silu", pre=s["pre"])
        m = ag.gemm_bias_act(s["h"], self.W2)
        s["y2"] = ag.layer_norm(m, self.g2, self.c2, residual=s["r"], h=s["s"], mean=s["mean2"], rstd=s["rstd2"])
        s["loss"], s["lse"] = ag.gemm_xent(s["y2"], self.V, targets)
        return s

    def backward(self, s, targets, dloss):
        d = {}
        dy, d["V"] = ag.gemm_xent_bwd(dloss, s["y2"], self.V, targets, s["lse"])
        ds, d["g2"], d["c2"] = ag.layer_norm_bwd(dy, s["s"], s["mean2"], s["rstd2"], weight=self.g2)
        dh, d["W2"], _ = ag.gemm_bias_act_bwd(ds, s["h"], self.W2, need_dbias=False)
        dy, d["W1"], d["b1"] = ag.gemm_bias_act_bwd(dh, s["y1"], self.W1, act="silu", pre=s["pre"])
        dr, d["g1"], d["c1"] = ag.layer_norm_bwd(dy, s["r"], s["mean1"], s["rstd1"], weight=self.g1, dh=ds)
        _, d["W0"], _ = ag.gemm_bias_act_bwd(dr, s["a"], self.W0, need_dA=False, need_dbias=False)
        return d

    def update(self, d, rate, decay=0.9):
        """Moves the parameters; returns the orthogonalised updates."""
        moves = {}
        for name, grad in d.items():
            p = self.parameters()[name]
            if name in self.momenta:
                m = self.momenta[name].mul_(decay).add_(grad)
                moves[name] = ag.newton_schulz(m)
                # an entry's size as that of a square matrix of the rows
                p.sub_(moves[name], alpha=0.1 * rate * max(1.0, p.shape[0] / p.shape[1]) ** 0.5)
            else:
                p.sub_(grad, alpha=rate)
        return moves

    def step(self, shards, targets, rate):
        dloss = (targets >= 0).float()
        dloss /= dloss.sum().clamp(min=1)
        s = self.forward(shards, targets)
        self.update(self.backward(s, targets, dloss), rate)
        return (s["loss"] * dloss).sum()


def main(steps=8):
    model, (shards, targets) = Model(), batch()
    losses = [float(x) for x in [model.step(shards, targets, rate=0.3) for _ in range(steps)]]
    print("mean loss by step:", " ".join("%.3f" % x for x in losses))
    return losses


if __name__ == "__main__":
    main()
