"""The example's training step: its gradients against differentiation in float64, and its loss going down."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def reference_gradients(model, shards, targets, order, ends, dloss):
    p = {k: v.double().requires_grad_(True) for k, v in model.parameters().items()}
    x = torch.cat(shards).double() @ p["W0"].t()
    h = x @ p["W1"].t() + p["b1"]
    y = (h * torch.sigmoid(h)) @ p["W2"].t() + x
    rows, z, lo = y[order], [], 0
    for e, hi in enumerate(ends.tolist()):
        z.append(rows[lo:hi] @ p["We"][e].t())
        lo = hi
    u = y.index_add(0, order, torch.cat(z))
    logits = u @ p["V"].t()
    has = targets >= 0
    hit = logits.gather(1, torch.where(has, targets, 0).unsqueeze(1)).squeeze(1)
    ((torch.logsumexp(logits, 1) - hit) * torch.where(has, dloss, 0.0)).sum().backward()
    return {k: v.grad for k, v in p.items()}


def test_gradients_of_the_step():
    import lm_step
    model, (shards, targets) = lm_step.Model(), lm_step.batch()
    dloss = torch.full((len(targets),), 1.0 / len(targets), device="cuda")
    s = model.forward(shards, targets)
    got = model.backward(s, targets, dloss)
    want = reference_gradients(model, shards, targets, s["order"], s["ends"], dloss)
    for name, g in got.items():
        off = float((g.double() - want[name]).norm() / want[name].norm())
        # at most sixteen tensors on a parameter's path are rounded to bf16, each off by 2^-8 of its size at most
        # and, in the norm, carried on by products whose weights have norms of about one
        assert off <= 16 * 2.0 ** -8, (name, off)


def test_loss_goes_down():
    import lm_step
    losses = lm_step.main(steps=6)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
