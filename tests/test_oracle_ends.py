"""The oracle of the router's losses and of the head's log probabilities against hand values, brute force
and differences."""
import math

import numpy as np
import pytest

from oracle import ends as O


def test_balance_loss_by_hand():
    # two tokens, two experts, k = 1: p = (3/4, 1/4) and (1/2, 1/2); both chose expert 0
    z = np.log(np.array([[3.0, 1.0], [1.0, 1.0]]))
    loss, counts, sums, tokens = O.balance_loss(z, np.array([[0], [0]], np.int32))
    assert counts.tolist() == [[2, 0]] and tokens.tolist() == [2]
    assert np.allclose(sums, [[1.25, 0.75]])
    assert math.isclose(loss[0], 2 / (1 * 4) * (2 * 1.25))
    # the same share for everyone: 1
    assert math.isclose(O.balance_loss(np.zeros((4, 4)), np.arange(4, dtype=np.int32)[:, None])[0][0], 1.0)


def test_sequences_and_padding_are_batches_of_their_own():
    rng = np.random.default_rng(1)
    z, ids = rng.normal(size=(20, 5)), rng.integers(0, 5, (20, 2)).astype(np.int32)
    valid = rng.random(20) < 0.7
    cuts = np.array([0, 7, 7, 18], np.int32)
    loss, counts, sums, tokens = O.balance_loss(z, ids, cuts, valid)
    for s in range(3):
        t = [i for i in range(cuts[s], cuts[s + 1]) if valid[i]]
        one = O.balance_loss(z[t], ids[t]) if t else (np.zeros(1), np.zeros((1, 5)), np.zeros((1, 5)), np.zeros(1))
        for got, want in zip((loss, counts, sums, tokens), one):
            assert np.allclose(got[s], want[0])


@pytest.mark.parametrize("renormalize", [True, False])
def test_router_gradient_against_differences(renormalize):
    rng = np.random.default_rng(2)
    T, E, k = 9, 6, 3
    z = rng.normal(size=(T, E))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[4] = [2, 2, 5]                                  # an id twice
    ids[5, 0] = -1                                      # no expert
    dw, dl, cuts = rng.normal(size=(T, k)), rng.normal(size=2), np.array([0, 5, 8], np.int32)
    valid = np.arange(T) != 3
    _, counts, _, tokens = O.balance_loss(z, ids, cuts, valid)
    d, mag = O.router_backward(z, ids, dw, renormalize, dl, counts, tokens, cuts, valid)
    assert (np.abs(d) <= mag + 1e-15).all()

    def f(v):
        return (O.balance_loss(v, ids, cuts, valid)[0] * dl).sum() + (O.route_weights(v, ids, renormalize) * dw).sum()

    for t in range(T):
        for e in range(E):
            h = np.zeros_like(z)
            h[t, e] = 1e-5
            assert abs((f(z + h) - f(z - h)) / 2e-5 - d[t, e]) < 1e-8


def test_head_gradients_against_differences():
    rng = np.random.default_rng(3)
    T, V, H = 4, 7, 5
    x, w = rng.normal(size=(T, H)), rng.normal(size=(V, H))
    y = np.array([3, -100, 6, 0])
    g, h = rng.normal(size=T), rng.normal(size=T)
    dx, dw, _ = O.head_logprobs_backward(x, w, y, g, h, 1.3)

    def f(x, w):
        out = O.head_logprobs(x, w, y, 1.3)
        return (out["logprob"] * g).sum() + (out["entropy"] * h).sum()

    for which, grad in ((0, dx), (1, dw)):
        for i in np.ndindex(grad.shape):
            a, b = [x.copy(), w.copy()], [x.copy(), w.copy()]
            a[which][i] += 1e-5
            b[which][i] -= 1e-5
            assert abs((f(*a) - f(*b)) / 2e-5 - grad[i]) < 1e-8
