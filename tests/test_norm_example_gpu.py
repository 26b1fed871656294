"""The pre-norm example: its gradients against differentiation in float64, its updates against the steps in float64, and that
a step runs the same on a graph's replays."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def reference_gradients(model, shards, targets, dloss):
    p = {k: v.double().requires_grad_(True) for k, v in model.parameters().items()}
    norm = torch.nn.functional.layer_norm
    r = torch.cat(shards).double() @ p["W0"].t()
    h = norm(r, r.shape[1:], p["g1"], p["c1"], 1e-5) @ p["W1"].t() + p["b1"]
    s = r + (h * torch.sigmoid(h)) @ p["W2"].t()
    logits = norm(s, s.shape[1:], p["g2"], p["c2"], 1e-5) @ p["V"].t()
    has = targets >= 0
    hit = logits.gather(1, torch.where(has, targets, 0).unsqueeze(1)).squeeze(1)
    ((torch.logsumexp(logits, 1) - hit) * torch.where(has, dloss, 0.0)).sum().backward()
    return {k: v.grad for k, v in p.items()}


def test_gradients_and_updates():
    import norm_step
    model, (shards, targets) = norm_step.Model(), norm_step.batch()
    # weights and biases of the norms that are not one and zero
    g = torch.Generator(device="cuda").manual_seed(3)
    for name in ("g1", "c1", "g2", "c2", "b1"):
        p = model.parameters()[name]
        p.add_(torch.randn(p.shape, generator=g, device="cuda").to(p.dtype), alpha=0.1)
    dloss = torch.full((len(targets),), 1.0 / len(targets), device="cuda")
    s = model.forward(shards, targets)
    got = model.backward(s, targets, dloss)
    want = reference_gradients(model, shards, targets, dloss)
    for name, grad in got.items():
        off = float((grad.double() - want[name]).norm() / want[name].norm())
        print(name, "%.2e" % off, flush=True)
        # at most sixteen tensors on a parameter's path are rounded to bf16, each off by 2^-8 of its size at most and, in the
        # norm, carried on by products whose weights have norms of about one
        assert off <= 16 * 2.0 ** -8, (name, off)
    from test_lm_ortho_gpu import OFF, exact, off
    before = {k: v.clone() for k, v in model.parameters().items()}
    for name, move in model.update(got, rate=0.1).items():
        assert off(move, exact(model.momenta[name])) <= OFF, name
        assert not torch.equal(model.parameters()[name], before[name])


def test_example_runs():
    import norm_step
    losses = norm_step.main(steps=3)
    assert len(losses) == 3 and all(x == x and 0 < x < 20 for x in losses)


def test_a_step_in_a_graph():
    """Forward, backward and the updates' products captured together: every replay's gradients and updates as an eager step's."""
    import norm_step
    model, (shards, targets) = norm_step.Model(), norm_step.batch()
    dloss = torch.full((len(targets),), 1.0 / len(targets), device="cuda")
    r = torch.cat(shards)
    import allgather_gemm_amd as ag

    def step():
        mean, rstd = torch.empty(2, r.shape[0], device="cuda")
        y = ag.layer_norm(r, model.g1, model.c1, mean=mean, rstd=rstd)
        loss, lse = ag.gemm_xent(y, model.V, targets)
        dy, dV = ag.gemm_xent_bwd(dloss, y, model.V, targets, lse)
        dr, dg, dc = ag.layer_norm_bwd(dy, r, mean, rstd, weight=model.g1)
        return loss, dr, dg, dc, ag.newton_schulz(dV), ag.newton_schulz(dr.t().contiguous())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    for i in range(4):
        r.copy_(torch.randn(r.shape, generator=torch.Generator().manual_seed(i)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, u in zip(out, step()):
            assert torch.equal(t, u), i
