"""Float64 oracle of the operators around the expert block in a learner's step: token log
probabilities with entropy and top alternatives, distillation from a teacher's top entries,
and their gradients.  Formulas only, row by row, with no regard for cancellation beyond what
float64 leaves; -inf logits are excluded tokens."""
from __future__ import annotations

import numpy as np


def softmax_stats(c):
    """(ln p, p, lse) of rows of scaled logits; an all-excluded row has lse = -inf, p = 0."""
    c = np.asarray(c, np.float64)
    m = c.max(1, keepdims=True)
    empty = np.isneginf(m)
    m0 = np.where(empty, 0.0, m)
    with np.errstate(divide="ignore"):
        ln_s = np.log(np.exp(c - m0).sum(1))
    # (c - m) - ln s, not c - lse: lse of a row of the type's lowest value is that value
    lp = np.where(np.isneginf(c), -np.inf, (c - m0) - np.where(empty[:, 0], 0.0, ln_s)[:, None])
    return lp, np.exp(lp), m0[:, 0] + ln_s


def _plogp(p, lp):
    return np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0)


def token_logprobs(z, targets=None, scale=1.0, k=0, ignore=-100):
    z = np.asarray(z, np.float64)
    T, V = z.shape
    lp, p, lse = softmax_stats(z * scale)
    ent = -_plogp(p, lp).sum(1)
    skip = np.zeros(T, bool) if targets is None else targets == ignore
    out = dict(lse=np.where(skip, 0.0, lse), entropy=np.where(skip, 0.0, ent))
    if targets is not None:
        at = lp[np.arange(T), np.clip(targets, 0, V - 1)]
        out["logprob"] = np.where(skip, 0.0, at)
    if k:
        order = np.argsort(-z, axis=1, kind="stable")[:, :k]
        val = np.take_along_axis(lp, order, 1)
        none = np.isneginf(np.take_along_axis(z, order, 1)) | skip[:, None]
        out["top_logprob"] = np.where(none, -np.inf, val)
        out["top_ids"] = np.where(none, -1, order).astype(np.int32)
    return out


def token_logprobs_backward(z, targets=None, dlogprob=None, dentropy=None, scale=1.0, ignore=-100):
    z = np.asarray(z, np.float64)
    T, V = z.shape
    lp, p, _ = softmax_stats(z * scale)
    d = np.zeros_like(z)
    if dlogprob is not None:
        ok = (targets >= 0) & (targets < V)
        g = np.where(ok, np.asarray(dlogprob, np.float64), 0.0)
        d -= g[:, None] * p
        d[np.arange(T)[ok], targets[ok]] += g[ok]
    if dentropy is not None:
        ent = -_plogp(p, lp).sum(1)
        d -= np.asarray(dentropy, np.float64)[:, None] * (_plogp(p, lp) + p * ent[:, None])
    d[np.isneginf(z)] = 0.0
    if targets is not None:
        d[targets == ignore] = 0.0
    return d * scale


def distill(z, ids, values, tail=True, scale=1.0):
    """(loss, dloss/dz, lse) of rows; ids of -1 are empty places."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    lp, p, lse = softmax_stats(z * scale)
    loss, grad = np.zeros(T), np.zeros_like(z)
    for t in range(T):
        live = ids[t] >= 0
        j, v = ids[t][live], np.asarray(values[t], np.float64)[live]
        if j.size == 0 or (not tail and np.all(np.isneginf(v))):
            lse[t] = 0.0
            continue
        q = np.exp(v) if tail else np.exp(v - v.max()) / np.exp(v - v.max()).sum()
        on = q > 0
        loss[t] = np.sum(q[on] * (np.log(q[on]) - lp[t, j[on]]))
        mass = q.sum()      # the teacher's mass that the loss counts
        if tail:
            listed = np.zeros(V, bool)
            listed[j] = True
            pr = p[t][~listed].sum()
            qr = max(0.0, 1.0 - q.sum())
            if pr > 0 and qr > 0:
                loss[t] += qr * (np.log(qr) - np.log(pr))
                grad[t][~listed] -= qr * p[t][~listed] / pr
                mass += qr
        grad[t] += mass * p[t]
        grad[t][j] -= q
    grad[np.isneginf(z)] = 0.0
    return loss, grad * scale, lse


def gate_rows(gate, T):
    """The gate as [T, 1] or [T, H]: None, one number a row, or rows that serve T / G rows each."""
    if gate is None:
        return np.ones((T, 1))
    gate = np.asarray(gate, np.float64)
    return gate[:, None] if gate.ndim == 1 else np.repeat(gate, T // gate.shape[0], axis=0)


def rstd(x, eps):
    x = np.asarray(x, np.float64)
    return 1.0 / np.sqrt((x * x).mean(1) + eps)


def norm_out(x, y, weight, gate=None, alpha=1.0, eps=1e-6):
    y = np.asarray(y, np.float64)
    return alpha * np.asarray(x, np.float64) + gate_rows(gate, y.shape[0]) * (y * rstd(y, eps)[:, None] * weight)


def norm_backward(du, x, r):
    """Gradient at x of xhat = x r(x), for the gradient du at xhat, with r = rstd(x) given."""
    xhat = x * r[:, None]
    return r[:, None] * (du - xhat * (du * xhat).mean(1, keepdims=True))


def norm_out_backward(dr, y, rstd_y, weight, gate=None, alpha=1.0, dn=None, r=None, rstd_r=None, next_weight=None):
    """(dx, dy, dweight, dgate or None, dnext or None)."""
    T, H = y.shape
    d = np.zeros((T, H)) if dr is None else np.asarray(dr, np.float64)
    dnext = dgate = None
    if dn is not None:
        d = d + norm_backward(dn * next_weight, r, rstd_r)
        dnext = (dn * r * rstd_r[:, None]).sum(0)
    g, yhat = gate_rows(gate, T), y * rstd_y[:, None]
    dy = norm_backward(d * g * weight, y, rstd_y)
    if gate is not None:
        full = d * weight * yhat
        dgate = full.sum(1) if np.ndim(gate) == 1 else full.reshape(len(gate), -1, H).sum(1)
    return alpha * d, dy, (d * g * yhat).sum(0), dgate, dnext
