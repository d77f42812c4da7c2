"""The learner's step of examples/router_head_step.py: the router's losses, the experts and the head in one path.
It runs, and its gradients of the router and the head are those of the formulas in float64 from the step's own
inputs to them."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import ends as O

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().cpu().double().numpy()


def test_runs(cuda_lib):
    import router_head_step
    losses = router_head_step.run(steps=3)
    assert len(losses) == 3 and all(np.isfinite(losses))


def test_gradients_of_the_router_and_the_head(cuda_lib):
    import router_head_step as M
    from nvfp4_w4a4_moe_quantize_gb300 import synthetic as S
    shape, V = S.WORKLOADS["tiny"], 1031
    learner = M.Learner(shape, V)
    targets, sequences = M.batch(shape, V)
    loss, bal, counts, grads, q = learner.step(targets, sequences)
    y, valid, cuts = targets.cpu().numpy(), q["valid"].cpu().numpy(), sequences.cpu().numpy()
    # the head: every element's d is off by half a BF16 step and the result again, 2^-8 each of the magnitudes
    x, w = f64(q["h"]), f64(q["head"])
    g = -valid.astype(np.float64) / valid.sum()
    want = O.head_logprobs(x, w, y)
    assert abs(loss.item() - float((want["logprob"] * g).sum())) < 1e-4
    _, dhead, d = O.head_logprobs_backward(x, w, y, g)
    tol = 2.0 ** -8 * (1.1 * np.abs(d).T @ np.abs(x) + np.abs(dhead)) + 1e-9
    assert (np.abs(f64(grads["head"]) - dhead) <= tol).all()
    # the router: float32 throughout; the products of its matrix are torch's own, 2^-17 of the magnitudes
    z, ids, n = f64(q["logits"]), q["ids"].cpu().numpy(), f64(q["n"])
    wl, wc, _, wt = O.balance_loss(z, ids, cuts, valid)
    assert np.abs(f64(bal) - wl).max() < 1e-5 and np.array_equal(counts.cpu().numpy(), wc)
    dz, mag = O.router_backward(z, ids, f64(q["dw"]), True, f64(q["dbal"]), wc, wt, cuts, valid)
    err = np.abs(f64(grads["router"]) - dz.T @ n)
    assert (err <= 2.0 ** -15 * (mag.T @ np.abs(n)) + 1e-12).all()
    # and its directional difference
    v = np.random.default_rng(0).normal(size=z.shape)

    def f(t):
        c = O.balance_loss(z + t * v, ids, cuts, valid)[0]
        return (c * f64(q["dbal"])).sum() + (O.route_weights(z + t * v, ids) * f64(q["dw"])).sum()

    assert abs((f(1e-5) - f(-1e-5)) / 2e-5 - (dz * v).sum()) < 1e-6 * np.abs(dz * v).sum() + 1e-12
