"""Float64 oracle of the losses at the two ends of a learner's step: the router's balance loss with the
gradient of its logits, and the log probabilities from hidden rows and the head's weight with theirs.
Formulas only, sequence by sequence and row by row."""
from __future__ import annotations

import numpy as np

from .learner import softmax_stats, token_logprobs, token_logprobs_backward


def _members(T, sequences, valid):
    """The token numbers of every sequence that count."""
    bounds = [0, T] if sequences is None else [int(v) for v in sequences]
    keep = np.ones(T, bool) if valid is None else np.asarray(valid) != 0
    return [np.array([t for t in range(a, b) if keep[t]], np.int64) for a, b in zip(bounds[:-1], bounds[1:])]


def balance_loss(z, ids, sequences=None, valid=None):
    """loss [S], counts [S, E], sums of probabilities [S, E], tokens [S]; ids outside [0, E) count nowhere."""
    z = np.asarray(z, np.float64)
    E, k = z.shape[1], ids.shape[1]
    loss, counts, sums, tokens = [], [], [], []
    for t in _members(z.shape[0], sequences, valid):
        p = softmax_stats(z[t])[1] if t.size else np.zeros((0, E))
        chosen = ids[t].reshape(-1)
        c = np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
        P, n = p.sum(0), t.size
        loss.append(E / (k * n * n) * float((c * P).sum()) if n else 0.0)
        counts.append(c)
        sums.append(P)
        tokens.append(n)
    return np.array(loss), np.array(counts, np.int32), np.array(sums), np.array(tokens, np.int32)


def route_weights(z, ids, renormalize=True):
    """w [T, k] of the chosen ids (0 for an id outside [0, E))."""
    z = np.asarray(z, np.float64)
    ok = (ids >= 0) & (ids < z.shape[1])
    at = np.where(ok, np.take_along_axis(z, np.clip(ids, 0, z.shape[1] - 1), 1), -np.inf)
    if renormalize:
        return softmax_stats(at)[1]
    return np.where(ok, np.take_along_axis(softmax_stats(z)[1], np.clip(ids, 0, z.shape[1] - 1), 1), 0.0)


def router_backward(z, ids, dweights=None, renormalize=True, dloss=None, counts=None, tokens=None, sequences=None,
                    valid=None):
    """(dlogits [T, E], the sum of the magnitudes that it is made of [T, E])."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    k = ids.shape[1]
    p = softmax_stats(z)[1]
    d, mag = np.zeros_like(p), np.zeros_like(p)
    if dloss is not None:
        for s, t in enumerate(_members(T, sequences, valid)):
            n = max(int(tokens[s]), 1)
            a = float(dloss[s]) * E * np.asarray(counts[s], np.float64) / (k * n * n)
            dot = (p[t] * a).sum(1, keepdims=True)
            d[t] += p[t] * (a - dot)
            mag[t] += p[t] * (np.abs(a) + np.abs(dot))
    if dweights is not None:
        w, dw = route_weights(z, ids, renormalize), np.asarray(dweights, np.float64)
        dot, adot = (w * dw).sum(1, keepdims=True), np.abs(w * dw).sum(1, keepdims=True)
        g = w * (dw - dot) if renormalize else w * dw
        ag = w * (np.abs(dw) + adot)
        for t in range(T):
            for j in range(k):
                if 0 <= ids[t, j] < E:
                    d[t, ids[t, j]] += g[t, j]
                    mag[t, ids[t, j]] += ag[t, j]
        if not renormalize:
            d -= p * dot
            mag += p * adot
    return d, mag


def head_logits(hidden, weight):
    return np.asarray(hidden, np.float64) @ np.asarray(weight, np.float64).T


def head_logprobs(hidden, weight, targets=None, scale=1.0, ignore=-100):
    """lse, entropy and (with targets) logprob of the rows, as token_logprobs of the logits."""
    return token_logprobs(head_logits(hidden, weight), targets, scale, ignore=ignore)


def head_logprobs_backward(hidden, weight, targets=None, dlogprob=None, dentropy=None, scale=1.0, ignore=-100):
    """(dhidden [T, H], dweight [V, H], d [T, V]) with d the gradient by the logits hidden @ weight^T."""
    x, w = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    d = token_logprobs_backward(head_logits(x, w), targets, dlogprob, dentropy, scale, ignore)
    return d @ w, d.T @ x, d
