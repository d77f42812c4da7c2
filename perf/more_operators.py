"""Measured cases of the losses at the two ends of a learner's step, with their gradients.

* ``balance``:        the router's balance loss and per-expert counts of every sequence.
* ``router_backward``: the gradient of the router's logits: that of the balance loss and that of
  the routing weights, in one pass.
* ``head``:           log probabilities of given tokens (the cross entropy, negated) and the
  entropy, from hidden rows and the head's weight, the logits never stored.
* ``head_backward``:  their gradients by the hidden rows and by the weight.

``own`` selects the framework's kernels; otherwise ``run`` computes the plain form:
elementary torch operations in float32 (long sums of probabilities in float64), each output
rounded once.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
IGNORE = -100
MOST = 8192 * 131072 * 2048      # rows x vocabulary x width of the largest head case


def listed():
    return [
        # a handful of tokens on a small router (latency counts)
        dict(name="balance_small", op="balance", T=64, E=8, k=2, S=1, dtype="f32", pad=0, masked=0.0),
        # the expert block's learner batch, one balance loss over all of it
        dict(name="balance_learner", op="balance", T=32768, E=128, k=8, S=1, dtype="f32", pad=0, masked=0.0),
        # packed sequences of ragged lengths, padding tokens inside and behind them, an odd number
        # of experts, half-precision logits in padded storage
        dict(name="balance_packed_odd", op="balance", T=10007, E=61, k=4, S=37, dtype="bf16", pad=3, masked=0.2),
        # the learner batch's router gradient: routing weights and balance loss
        dict(name="router_backward_learner", op="router_backward", T=32768, E=128, k=8, S=1, dtype="f32", pad=0,
             masked=0.0, renormalize=True, weights=True, balance=True),
        # packed sequences, more experts than a power of two, plain probabilities as weights
        dict(name="router_backward_odd", op="router_backward", T=4999, E=257, k=6, S=19, dtype="f16", pad=0,
             masked=0.1, renormalize=False, weights=True, balance=True),
        # one token of a rollout scored against the whole vocabulary: the weight is read once
        dict(name="head_decode", op="head", T=1, V=131072, H=2048, dtype="bf16", pad=0, scale=1.0, ignored=0.0,
             entropy=True),
        # a short rollout, an odd vocabulary, a sampling temperature, finished sequences as ignored
        # rows, padded storage
        dict(name="head_rollout_odd", op="head", T=96, V=50021, H=1032, dtype="f16", pad=8, scale=1.4, ignored=0.2,
             entropy=False),
        # the learner's forward over a micro-batch of packed sequences
        dict(name="head_learner", op="head", T=8192, V=131072, H=2048, dtype="bf16", pad=0, scale=1.0, ignored=0.1,
             entropy=True),
        # gradients of a few rows: the weight's gradient is the traffic
        dict(name="head_backward_short", op="head_backward", T=48, V=131072, H=2048, dtype="bf16", pad=0, scale=1.0,
             ignored=0.0, entropy=False),
        # an odd vocabulary and odd numbers of rows in half precision with a loss scale and an
        # entropy bonus
        dict(name="head_backward_odd", op="head_backward", T=1001, V=50021, H=1032, dtype="f16", pad=8, scale=0.8,
             ignored=0.3, entropy=True),
        # the learner's backward of a micro-batch
        dict(name="head_backward_learner", op="head_backward", T=8192, V=131072, H=2048, dtype="bf16", pad=0,
             scale=1.0, ignored=0.1, entropy=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "router_backward", "head", "head", "head_backward", "head_backward"])
    if not op.startswith("head"):
        E = rng.choice([8, 16, 64, 128, 256, _log_int(rng, 4, 1024), _log_int(rng, 4, 1024)])
        T = _log_int(rng, 1, max(1, min(32768, 32768 * 128 // E)))
        case = dict(op=op, T=T, E=E, k=min(E, _log_int(rng, 1, 16)), S=min(T, rng.choice([1, 1, _log_int(rng, 1, 64)])),
                    dtype=rng.choice(["f32", "f32", "bf16", "f16"]), pad=rng.choice([0, 0, rng.randint(1, 16)]),
                    masked=rng.choice([0.0, 0.0, 0.2]))
        if op == "router_backward":
            case["renormalize"] = rng.random() < 0.6
            case["weights"], case["balance"] = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return case
    V = _log_int(rng, 1000, 262144)
    if rng.random() < 0.5:
        V = V // 64 * 64
    H = _log_int(rng, 32, 512) * 8
    T = _log_int(rng, 1, max(1, min(16384, MOST // 2 // (V * H))))
    return dict(op=op, T=T, V=V, H=H, dtype=rng.choice(["bf16", "bf16", "f16"]), pad=rng.choice([0, 0, 8, 64]),
                scale=rng.choice([1.0, 1.0, 0.8, 1.4]), ignored=rng.choice([0.0, 0.1, 0.5]),
                entropy=rng.random() < 0.5)


# ------------------------------------------------------------------------------- inputs

def _router_state(case, gen):
    """Router logits with popular and unpopular experts, the top-k of every row, and sequences:
    ragged lengths, a few tokens behind the last one, padding tokens inside."""
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    z = 1.5 * torch.randn(T, E + case["pad"], generator=gen, device="cuda")
    z = (z + 0.8 * torch.randn(E + case["pad"], generator=gen, device="cuda")).to(DTYPES[case["dtype"]])[:, :E]
    state = dict(case=case, logits=z, ids=z.float().topk(k, dim=1).indices.to(torch.int32),
                 sequences=None, valid=None)
    if S > 1:
        cuts = torch.rand(S, generator=gen, device="cuda").sort().values
        end = int(T - T // 50)
        offsets = torch.cat([torch.zeros(1, device="cuda"), (cuts[1:] * end).round(), torch.full((1,), float(end),
                                                                                                  device="cuda")])
        state["sequences"] = offsets.to(torch.int32)
    if case["masked"] > 0.0:
        state["valid"] = torch.rand(T, generator=gen, device="cuda") >= case["masked"]
    return state


def _head_inputs(case, gen):
    """Hidden rows of unit variance and a head whose logits have a deviation of about 2; every
    row leans towards its token, as a trained model's do.  Storage may be padded."""
    T, V, H, dt = case["T"], case["V"], case["H"], DTYPES[case["dtype"]]
    w = (torch.randn(V, H + case["pad"], generator=gen, device="cuda") * (2.0 / math.sqrt(H))).to(dt)[:, :H]
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    lean = (2.0 + 8.0 * torch.rand(T, 1, generator=gen, device="cuda")) / 4.0
    x = torch.randn(T, H + case["pad"], generator=gen, device="cuda")
    x[:, :H] += lean * w[y].float()
    skip = torch.rand(T, generator=gen, device="cuda") < case["ignored"]
    return x.to(dt)[:, :H], w, torch.where(skip, torch.full_like(y, IGNORE), y).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if not case["op"].startswith("head"):
        state = _router_state(case, gen)
        if case["op"] == "router_backward":
            # what the forward leaves behind, and the gradients that arrive
            _, counts, _, tokens = _balance_plain(state)
            state["dweights"] = torch.randn(case["T"], case["k"], generator=gen, device="cuda") / case["T"]
            state["dloss"] = 0.01 * (1.0 + torch.rand(case["S"], generator=gen, device="cuda"))
            state["counts"], state["tokens"] = counts, tokens
            if case["dtype"] == "f16":       # half-precision gradients travel with a loss scale
                state["dweights"] *= 4096.0
                state["dloss"] *= 4096.0
            if not case["weights"]:
                state["dweights"] = None
            if not case["balance"]:
                state["dloss"] = state["counts"] = state["tokens"] = None
        return state
    x, w, y = _head_inputs(case, gen)
    state = dict(case=case, hidden=x, weight=w, targets=y)
    if case["op"] == "head_backward":
        T = case["T"]
        _, state["lse"], entropy = _head_plain(state)
        unit = (1024.0 if case["dtype"] == "f16" else 1.0) / math.sqrt(T)
        state["dlogprob"] = torch.randn(T, generator=gen, device="cuda") * unit
        state["entropy"] = entropy if case["entropy"] else None
        state["dentropy"] = torch.full((T,), -0.01 * unit, device="cuda") if case["entropy"] else None
    return state


# ------------------------------------------------------------------------------- plain forms

def _members(state):
    """Of every token its sequence (S: none) and whether it counts."""
    case, T = state["case"], state["case"]["T"]
    place = torch.arange(T, device="cuda")
    if state["sequences"] is None:
        seq = torch.zeros(T, dtype=torch.int64, device="cuda")
    else:
        seq = (place[:, None] >= state["sequences"][None, 1:]).sum(1)
    live = seq < case["S"]
    if state["valid"] is not None:
        live = live & state["valid"]
    return torch.where(live, seq, torch.full_like(seq, case["S"])), live


def _softmax_plain(z):
    e = (z.float() - z.float().amax(1, keepdim=True)).exp()
    return e / e.sum(1, keepdim=True)


def _balance_plain(state):
    """loss [S], counts [S, E], sums of probabilities [S, E], tokens [S]."""
    case = state["case"]
    S, E, k = case["S"], case["E"], case["k"]
    seq, live = _members(state)
    p = _softmax_plain(state["logits"])
    sums = torch.zeros(S + 1, E, dtype=torch.float64, device="cuda").index_add_(0, seq, p.double())[:S]
    places = seq[:, None] * E + state["ids"].long()
    counts = torch.zeros((S + 1) * E, dtype=torch.int64, device="cuda").index_add_(
        0, places.reshape(-1), torch.ones_like(places.reshape(-1))).view(S + 1, E)[:S]
    tokens = torch.zeros(S + 1, dtype=torch.int64, device="cuda").index_add_(0, seq, torch.ones_like(seq))[:S]
    n = tokens.double().clamp(min=1.0)
    loss = E / k * (counts.double() * sums).sum(1) / (n * n)
    return loss.float(), counts.to(torch.int32), sums.float(), tokens.to(torch.int32)


def _router_backward_plain(state):
    case, z = state["case"], state["logits"]
    p = _softmax_plain(z)
    d = torch.zeros_like(p)
    if state["dloss"] is not None:
        seq, live = _members(state)
        n = state["tokens"].float().clamp(min=1.0)
        a = state["dloss"][:, None] * (case["E"] / case["k"]) * (state["counts"].float() / n[:, None]) / n[:, None]
        a = torch.cat([a, torch.zeros_like(a[:1])])[seq]
        d = p * (a - (p * a).sum(1, keepdim=True))
    if state["dweights"] is not None:
        ids, dw = state["ids"].long(), state["dweights"]
        if case["renormalize"]:
            w = _softmax_plain(z.float().gather(1, ids))
            d = d.scatter_add(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
        else:
            w = p.gather(1, ids)
            d = (d - p * (w * dw).sum(1, keepdim=True)).scatter_add(1, ids, w * dw)
    return d.to(z.dtype)


def _head_plain(state):
    """logprob, lse and entropy [T]."""
    y = state["targets"]
    c = (state["hidden"].float() @ state["weight"].float().t()) * state["case"]["scale"]
    m = c.amax(1, keepdim=True)
    lse = (c - m).exp().sum(1).log() + m.squeeze(1)
    c -= lse[:, None]                       # log probabilities
    logprob = c.gather(1, y.clamp(min=0).long()[:, None]).squeeze(1)
    entropy = -(c.exp() * c).sum(1)
    skip, zero = y == IGNORE, torch.zeros_like(lse)
    return torch.where(skip, zero, logprob), torch.where(skip, zero, lse), torch.where(skip, zero, entropy)


def _head_backward_plain(state):
    """Gradients by the hidden rows [T, H] and the weight [V, H]."""
    case, y = state["case"], state["targets"]
    x, w = state["hidden"].float(), state["weight"].float()
    c = (x @ w.t()) * case["scale"] - state["lse"][:, None]
    p = c.exp()
    g = state["dlogprob"][:, None]
    d = (-g) * p
    d.scatter_add_(1, y.clamp(min=0).long()[:, None], g)
    if case["entropy"]:
        d -= state["dentropy"][:, None] * p * (c + state["entropy"][:, None])
    d *= torch.where(y == IGNORE, torch.zeros_like(state["lse"]), torch.full_like(state["lse"], case["scale"]))[:, None]
    return (d @ w).to(state["hidden"].dtype), (d.t() @ x).to(state["weight"].dtype)


# ------------------------------------------------------------------------------- one pass

def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        import nvfp4_w4a4_moe_quantize_gb300 as lib
        if op == "balance":
            return lib.moe_balance_loss(state["logits"], state["ids"], sequences=state["sequences"],
                                        valid=state["valid"])
        if op == "router_backward":
            return lib.moe_router_backward(state["logits"], state["ids"], dweights=state["dweights"],
                                           renormalize=case["renormalize"], dloss=state["dloss"],
                                           counts=state["counts"], tokens=state["tokens"],
                                           sequences=state["sequences"], valid=state["valid"])
        if op == "head":
            return lib.head_logprobs(state["hidden"], state["weight"], state["targets"], scale=case["scale"],
                                     ignore_index=IGNORE, entropy=case["entropy"])[:3 if case["entropy"] else 2]
        return lib.head_logprobs_backward(state["hidden"], state["weight"], state["lse"], state["targets"],
                                          state["dlogprob"], entropy=state["entropy"], dentropy=state["dentropy"],
                                          scale=case["scale"], ignore_index=IGNORE)
    if op == "balance":
        return _balance_plain(state)
    if op == "router_backward":
        return _router_backward_plain(state)
    if op == "head":
        return _head_plain(state)[:3 if case["entropy"] else 2]
    return _head_backward_plain(state)


def work(case):
    T, e = case["T"], BYTES[case["dtype"]]
    if not case["op"].startswith("head"):
        E, k, S = case["E"], case["k"], case["S"]
        extra = (4 * (S + 1) if S > 1 else 0) + (T if case["masked"] > 0.0 else 0)
        if case["op"] == "balance":
            return {"bytes": T * E * e + 4 * T * k + 8 * S * E + 8 * S + extra, "flops": 5 * T * E}
        moved = 2 * T * E * e + 4 * T * k + (4 * T * k if case["weights"] else 0)
        if case["balance"]:
            moved += 4 * S * E + 8 * S + extra
        return {"bytes": moved, "flops": (4 + 4 * case["balance"]) * T * E + 8 * case["weights"] * T * k}
    V, H = case["V"], case["H"]
    rows = max(1, int(round(T * (1.0 - case["ignored"]))))     # rows that have a token to score
    if case["op"] == "head":
        return {"bytes": (rows + V) * H * e + 4 * T * (4 if case["entropy"] else 3), "flops": 2 * rows * V * H}
    # the logits again, then two products with their gradient
    return {"bytes": (rows + V + T + V) * H * e + 4 * T * (5 if case["entropy"] else 3), "flops": 6 * rows * V * H}


# ------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions in float64: sequence by sequence for the router, block of rows by block of
    rows for the head."""
    state = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(case, state)
    if case["op"] == "router_backward":
        return _exact_router_backward(case, state)
    # float64 products run at about one teraflop a second
    if 2.0 * case["T"] * case["V"] * case["H"] * (1 if case["op"] == "head" else 3) > 1.5e13:
        return None
    return _exact_head(case, state) if case["op"] == "head" else _exact_head_backward(case, state)


def _spans(case, state):
    """The token numbers of every sequence."""
    T = case["T"]
    bounds = [0, T] if state["sequences"] is None else state["sequences"].tolist()
    out = []
    for s in range(case["S"]):
        t = torch.arange(bounds[s], bounds[s + 1], device="cuda")
        out.append(t if state["valid"] is None else t[state["valid"][t]])
    return out


def _exact_balance(case, state):
    E, k = case["E"], case["k"]
    loss, counts, sums, tokens = [], [], [], []
    for t in _spans(case, state):
        p = torch.softmax(state["logits"][t].double(), 1)
        c = torch.bincount(state["ids"][t].long().reshape(-1), minlength=E)
        n = t.numel()
        share = c.double() / max(1, n * k)
        loss.append(E * (share * p.sum(0) / max(1, n)).sum())
        counts.append(c.to(torch.int32))
        sums.append(p.sum(0))
        tokens.append(n)
    return (torch.stack(loss), torch.stack(counts), torch.stack(sums),
            torch.tensor(tokens, dtype=torch.int32, device="cuda"))


def _exact_router_backward(case, state):
    """By the Jacobian of the softmax: dz = J^T dp, row by row through autograd in float64."""
    E, k = case["E"], case["k"]
    z = state["logits"].double().detach().requires_grad_()
    p = torch.softmax(z, 1)
    total = (p * 0.0).sum()
    if state["dloss"] is not None:
        for s, t in enumerate(_spans(case, state)):
            n = state["tokens"][s].double().clamp(min=1.0)
            share = state["counts"][s].double() / (k * n)
            total = total + state["dloss"][s].double() * E * (share * (p[t].sum(0) / n)).sum()
    if state["dweights"] is not None:
        picked = p.gather(1, state["ids"].long())
        if case["renormalize"]:
            picked = picked / picked.sum(1, keepdim=True)
        total = total + (picked * state["dweights"].double()).sum()
    return torch.autograd.grad(total, z)[0]


def _blocks(case):
    step = max(1, (1 << 28) // case["V"])
    return [(a, min(case["T"], a + step)) for a in range(0, case["T"], step)]


def _exact_head(case, state):
    w = state["weight"].double()
    logprob, lses, entropy = [], [], []
    for a, b in _blocks(case):
        y = state["targets"][a:b].long()
        lp = torch.log_softmax(state["hidden"][a:b].double() @ (w.t() * case["scale"]), 1)
        # lse from any token's logit and its log probability
        first = (state["hidden"][a:b].double() * w[0]).sum(1) * case["scale"]
        keep = (y != IGNORE).double()
        logprob.append(lp[torch.arange(b - a, device="cuda"), y.clamp(min=0)] * keep)
        lses.append((first - lp[:, 0]) * keep)
        entropy.append(-torch.xlogy(lp.exp(), lp.exp()).sum(1) * keep)
    out = (torch.cat(logprob), torch.cat(lses), torch.cat(entropy))
    return out if case["entropy"] else out[:2]


def _exact_head_backward(case, state):
    w = state["weight"].double()
    dx, dw = [], torch.zeros(case["V"], case["H"], dtype=torch.float64, device="cuda")
    for a, b in _blocks(case):
        x, y = state["hidden"][a:b].double(), state["targets"][a:b].long()
        lp = torch.log_softmax(x @ w.t() * case["scale"], 1)
        d = torch.softmax(lp, 1).neg()
        d[torch.arange(b - a, device="cuda"), y.clamp(min=0)] += 1.0
        d *= state["dlogprob"][a:b, None].double()
        if case["entropy"]:
            plogp = lp.exp() * lp
            d -= state["dentropy"][a:b, None].double() * (plogp - lp.exp() * plogp.sum(1, keepdim=True))
        d[y == IGNORE] = 0.0
        d *= case["scale"]
        dx.append(d @ w)
        dw += d.t() @ x
    return torch.cat(dx), dw
