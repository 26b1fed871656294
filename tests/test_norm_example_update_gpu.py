"""The pre-norm example's update: where each parameter goes, and what its momentum carries from step to step."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

from lm_reference import F, H, near  # noqa: E402

pytestmark = pytest.mark.gpu
RATE, DECAY = 0.3, 0.9


def gradients(model, batch):
    shards, targets = batch
    dloss = torch.full((len(targets),), 1.0 / len(targets), device="cuda")
    return model.backward(model.forward(shards, targets), targets, dloss)


def check_moved(before, after, alpha, move, name):
    """after = bf16(before - alpha move): the product and the difference in fp32, then one rounding."""
    want = before.double() - alpha * move.double()
    near(after, want, H * want.abs() * (1 + H) + 3 * F * (before.double().abs() + abs(alpha) * move.double().abs()), name)


def test_parameters_move_down_and_momenta_carry_on():
    import norm_step
    from ortho_reference import bound, exact, off, spectrum
    import allgather_gemm_amd as ag
    model, batch = norm_step.Model(), norm_step.batch()
    momenta = {k: torch.zeros(m.shape, dtype=torch.float64, device="cuda") for k, m in model.momenta.items()}
    assert set(momenta) == {"W0", "W1", "W2"}
    for step in range(3):
        grads = gradients(model, batch)
        before = {k: v.clone() for k, v in model.parameters().items()}
        assert set(grads) == set(before)
        moves = model.update(grads, RATE)
        assert set(moves) == set(momenta)
        for name, p in model.parameters().items():
            if name not in momenta:
                check_moved(before[name], p, RATE, grads[name], name)
                continue
            m = momenta[name]
            off_m = 2 * F * (DECAY * m.abs() + grads[name].double().abs()) + 3 * step * F * m.abs()
            m.mul_(DECAY).add_(grads[name].double())
            near(model.momenta[name], m, off_m, name)
            s, n = spectrum(model.momenta[name])
            o, most = off(moves[name], exact(model.momenta[name], ag.NEWTON_SCHULZ)), bound(s, n, ag.NEWTON_SCHULZ, True)
            print(step, name, "%.2e of %.2e" % (o, most), flush=True)
            assert o <= most, (name, o, most)
            check_moved(before[name], p, 0.1 * RATE * max(1.0, p.shape[0] / p.shape[1]) ** 0.5, moves[name], name)


def test_a_step_is_its_parts():
    """step() is forward, backward and update, with the loss and its gradient over the rows that have a target."""
    import norm_step
    one, two, (shards, targets) = norm_step.Model(), norm_step.Model(), norm_step.batch()
    for _ in range(2):
        loss = one.step(shards, targets, RATE)
        has = targets >= 0
        dloss = has.float() / has.sum()
        s = two.forward(shards, targets)
        two.update(two.backward(s, targets, dloss), RATE)
        assert abs(float(loss) - float(s["loss"][has].double().mean())) <= len(targets) * F * float(loss)
        for k, p in two.parameters().items():
            assert torch.equal(one.parameters()[k], p), k
        for k, m in two.momenta.items():
            assert torch.equal(one.momenta[k], m), k
