"""The float64 oracle of the learner's operators against closed forms and differences."""
import numpy as np
import pytest

from oracle import learner as O


def _rows(seed, T=4, V=23, masked=False):
    rng = np.random.default_rng(seed)
    z = rng.normal(0.0, 2.0, (T, V))
    if masked:
        z[rng.random((T, V)) < 0.3] = -np.inf
        z[:, :3] = rng.normal(0.0, 2.0, (T, 3))
    return z, rng


def test_uniform_row():
    r = O.token_logprobs(np.full((1, 16), 3.0), np.array([5]), k=3)
    np.testing.assert_allclose(r["logprob"], -np.log(16))
    np.testing.assert_allclose(r["entropy"], np.log(16))
    np.testing.assert_array_equal(r["top_ids"], [[0, 1, 2]])          # equal values by lower id


def test_excluded_and_empty_rows():
    z = np.full((2, 4), -np.inf)
    z[0, 2] = 1.5
    r = O.token_logprobs(z, np.array([2, 0]), k=2)
    assert r["logprob"][0] == 0 and r["entropy"][0] == 0 and r["lse"][0] == 1.5
    assert np.isneginf(r["lse"][1]) and np.isneginf(r["logprob"][1]) and r["entropy"][1] == 0
    np.testing.assert_array_equal(r["top_ids"], [[2, -1], [-1, -1]])


def _differences(f, z, h=1e-6):
    d = np.zeros_like(z)
    for i in np.ndindex(z.shape):
        if np.isneginf(z[i]):
            continue
        a, b = z.copy(), z.copy()
        a[i] += h
        b[i] -= h
        d[i] = (f(a) - f(b)) / (2 * h)
    return d


@pytest.mark.parametrize("masked", [False, True])
def test_logprob_gradient_by_differences(masked):
    z, rng = _rows(1, masked=masked)
    y = np.array([0, 1, -100, 2])
    g, h = rng.normal(size=4), rng.normal(size=4)

    def f(x):
        r = O.token_logprobs(x, y, scale=0.7)
        return np.sum(g * r["logprob"] + h * r["entropy"])

    np.testing.assert_allclose(O.token_logprobs_backward(z, y, g, h, scale=0.7), _differences(f, z), atol=1e-8)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_distill_gradient_by_differences(tail, masked):
    z, rng = _rows(2, masked=masked)
    ids = np.array([[0, 1, 2, -1], [2, 1, 0, -1], [-1] * 4, [1, -1, -1, -1]])
    v = np.log(rng.dirichlet(np.ones(6), 4)[:, :4])
    loss, grad, _ = O.distill(z, ids, v, tail, 1.3)
    assert loss[2] == 0 and not grad[2].any()
    np.testing.assert_allclose(grad, _differences(lambda x: O.distill(x, ids, v, tail, 1.3)[0].sum(), z), atol=1e-8)


def test_distill_is_zero_at_the_teacher():
    z, _ = _rows(3)
    lp, _, _ = O.softmax_stats(z)
    ids = np.argsort(-z, 1)[:, :5]
    v = np.take_along_axis(lp, ids, 1)
    loss, grad, _ = O.distill(z, ids, v, True)
    np.testing.assert_allclose(loss, 0.0, atol=1e-14)
    np.testing.assert_allclose(grad, 0.0, atol=1e-14)


@pytest.mark.parametrize("kind", ["none", "token", "rows"])
def test_norm_gradients_by_differences(kind):
    rng = np.random.default_rng(4)
    T, H, eps, alpha = 6, 5, 1e-3, 0.7
    x, y, w, wn = rng.normal(size=(T, H)), rng.normal(size=(T, H)), rng.normal(size=H), rng.normal(size=H)
    gate = {"none": None, "token": rng.normal(size=T), "rows": rng.normal(size=(3, H))}[kind]
    cr, cn = rng.normal(size=(T, H)), rng.normal(size=(T, H))

    def f(x=x, y=y, w=w, gate=gate, wn=wn):
        r = O.norm_out(x, y, w, gate, alpha, eps)
        return np.sum(cr * r) + np.sum(cn * r * O.rstd(r, eps)[:, None] * wn)

    r = O.norm_out(x, y, w, gate, alpha, eps)
    dx, dy, dw, dg, dnext = O.norm_out_backward(cr, y, O.rstd(y, eps), w, gate, alpha, cn, r, O.rstd(r, eps), wn)
    np.testing.assert_allclose(dx, _differences(lambda v: f(x=v), x), atol=1e-7)
    np.testing.assert_allclose(dy, _differences(lambda v: f(y=v), y), atol=1e-7)
    np.testing.assert_allclose(dw, _differences(lambda v: f(w=v), w), atol=1e-7)
    np.testing.assert_allclose(dnext, _differences(lambda v: f(wn=v), wn), atol=1e-7)
    if gate is not None:
        np.testing.assert_allclose(dg, _differences(lambda v: f(gate=v), gate), atol=1e-7)


def test_distill_gradient_where_the_masses_do_not_add_up_to_one():
    """With the tail: a mask that leaves the list alone while the list's mass is below one (nothing stands
    for the rest), a list of more than one, and both."""
    z, _ = _rows(5, T=4, V=9)
    z[[0, 2], 3:] = -np.inf
    z[0, :3] = [1.0, 2.0, 0.5]
    ids = np.tile([0, 1, 2], (4, 1))
    q = np.array([[0.4, 0.3, 0.1], [0.6, 0.5, 0.2], [0.6, 0.5, 0.2], [0.4, 0.3, 0.1]])
    grad = O.distill(z, ids, np.log(q), True, 1.3)[1]
    np.testing.assert_allclose(grad, _differences(lambda x: O.distill(x, ids, np.log(q), True, 1.3)[0].sum(), z),
                               atol=1e-8)
    np.testing.assert_allclose(grad.sum(1), 0.0, atol=1e-14)   # the loss does not change with a shift of the row
