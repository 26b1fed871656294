"""A training step of a small language model's block and head over row shards, with the library's operators alone:

    x = gather(shards) W0^T                                    ag_gemm
    h = silu(x W1^T + b1);  y = h W2^T + x                     gemm_bias_act
    z[t] = y[t] We[e(t)]^T,  u = y + z                         gemm_grouped, rows sorted by expert
    loss = cross entropy of u V^T against the next token       gemm_xent

and its gradients by the matching ..._bwd calls, followed by a step of gradient descent.  Nothing is copied to the
host inside a step: the experts' row counts stay on the device.

    python examples/lm_step.py            # prints the mean loss of each step
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import allgather_gemm_amd as ag  # noqa: E402

BF16 = torch.bfloat16


class Model:
    def __init__(self, width=256, hidden=512, experts=4, vocab=1003, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5).to(BF16)

        self.W0, self.W1, self.W2 = weight(width, width), weight(hidden, width), weight(width, hidden)
        self.b1 = torch.zeros(hidden, dtype=BF16, device="cuda")
        self.We, self.V = weight(experts, width, width), weight(vocab, width)
        self.router = weight(experts, width)          # fixed: which expert a row goes to

    def parameters(self):
        return {"W0": self.W0, "W1": self.W1, "b1": self.b1, "W2": self.W2, "We": self.We, "V": self.V}

    def forward(self, shards, targets):
        s = {}
        rows = sum(t.shape[0] for t in shards)
        s["a"] = torch.empty(rows, shards[0].shape[1], dtype=BF16, device="cuda")
        s["x"] = ag.ag_gemm(shards, self.W0, 128, a_out=s["a"])
        s["pre"] = torch.empty(rows, self.W1.shape[0], dtype=BF16, device="cuda")
        s["h"] = ag.gemm_bias_act(s["x"], self.W1, bias=self.b1, act="silu", pre=s["pre"])
        s["y"] = ag.gemm_bias_act(s["h"], self.W2, residual=s["x"])
        expert = ag.gemm_bias_act(s["y"], self.router).argmax(1)
        s["order"] = torch.sort(expert, stable=True).indices
        s["ends"] = torch.searchsorted(expert[s["order"]], torch.arange(1, self.We.shape[0] + 1, device="cuda"), out_int32=True)
        s["sorted"] = s["y"][s["order"]]
        z = ag.gemm_grouped(s["sorted"], self.We, s["ends"])
        s["u"] = s["y"].index_add(0, s["order"], z)   # each row once
        s["loss"], s["lse"] = ag.gemm_xent(s["u"], self.V, targets)
        return s

    def backward(self, s, targets, dloss):
        d = {}
        du, d["V"] = ag.gemm_xent_bwd(dloss, s["u"], self.V, targets, s["lse"])
        dsorted, d["We"] = ag.gemm_grouped_bwd(du[s["order"]], s["sorted"], self.We, s["ends"])
        dy = du.index_add(0, s["order"], dsorted)
        dh, d["W2"], _ = ag.gemm_bias_act_bwd(dy, s["h"], self.W2, need_dbias=False)
        dx, d["W1"], d["b1"] = ag.gemm_bias_act_bwd(dh, s["x"], self.W1, act="silu", pre=s["pre"])
        _, d["W0"], _ = ag.gemm_bias_act_bwd(dx + dy, s["a"], self.W0, need_dA=False, need_dbias=False)
        return d

    def step(self, shards, targets, rate):
        dloss = (targets >= 0).float()
        dloss /= dloss.sum().clamp(min=1)
        s = self.forward(shards, targets)
        for name, grad in self.backward(s, targets, dloss).items():
            self.parameters()[name].sub_(grad, alpha=rate)
        return (s["loss"] * dloss).sum()


def batch(ranks=4, rows=96, width=256, vocab=1003, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shards = [torch.randn(rows, width, generator=g, device="cuda").to(BF16) for _ in range(ranks)]
    targets = torch.randint(0, vocab, (ranks * rows,), generator=g, device="cuda")
    targets[::17] = -100                              # rows without a next token
    return shards, targets


def main(steps=8):
    model, (shards, targets) = Model(), batch()
    # small enough that the loss falls on every step whatever order the sums are taken in (at 1.0 it wanders near 0.03)
    losses = [model.step(shards, targets, rate=0.3) for _ in range(steps)]
    losses = [float(x) for x in losses]
    print("mean loss by step:", " ".join("%.3f" % x for x in losses))
    return losses


if __name__ == "__main__":
    main()
