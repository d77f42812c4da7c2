"""Measured cases of the operators around the expert block in a learner's step.

* ``logprobs``:  log probabilities of given tokens with entropy and top alternatives,
  forward and backward.
* ``distill``:   distillation from a teacher's top logits, loss alone or loss and gradient.
* ``norm``:      the RMS norms before and after the block, with its gate and residual scale,
  forward and backward.

``own`` selects the framework's kernels; otherwise ``run`` computes the plain form:
elementary torch operations in float32, each output rounded once.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
IGNORE = -100
EPS = 1e-6


def listed():
    return [
        # one sequence being decoded: the sampled token's log probability, the entropy and
        # the 20 best alternatives of one row (latency counts)
        dict(name="logprobs_decode", op="logprobs", T=1, V=131072, dtype="bf16", pad=0, top_k=20, scale=1.0,
             masked=0.0, ignored=0.0),
        # a rollout batch under a grammar mask, an odd vocabulary (rows of every alignment),
        # a sampling temperature, finished sequences as ignored rows
        dict(name="logprobs_rollout_odd", op="logprobs", T=96, V=50021, dtype="f16", pad=0, top_k=5, scale=1.4,
             masked=0.3, ignored=0.2),
        # the teacher's pass over a micro-batch, which keeps the 128 best tokens of each row
        dict(name="logprobs_teacher", op="logprobs", T=2048, V=131072, dtype="bf16", pad=0, top_k=128, scale=1.0,
             masked=0.0, ignored=0.0),
        # the learner's forward over a micro-batch of packed sequences
        dict(name="logprobs_learner", op="logprobs", T=8192, V=131072, dtype="bf16", pad=0, top_k=0, scale=1.0,
             masked=0.0, ignored=0.1),
        # the learner's backward of the same: a policy gradient and an entropy bonus
        dict(name="logprobs_learner_backward", op="logprobs_backward", T=8192, V=131072, dtype="bf16", pad=0, scale=1.0,
             masked=0.0, ignored=0.1, entropy=True),
        # evaluation of a student on a few rows of float32 logits in padded storage
        dict(name="distill_eval", op="distill", T=17, V=32003, dtype="f32", pad=61, K=16, tail=True, scale=1.0,
             masked=0.1, short=0.2, grad=False),
        # ragged teacher lists, half-precision logits of an odd vocabulary, renormalised teacher
        dict(name="distill_step_odd", op="distill", T=1000, V=50021, dtype="f16", pad=0, K=100, tail=False, scale=0.8,
             masked=0.0, short=0.5, grad=True),
        # the learner's distillation step: loss and gradient of a micro-batch
        dict(name="distill_step_learner", op="distill", T=8192, V=131072, dtype="bf16", pad=0, K=64, tail=True,
             scale=1.0, masked=0.0, short=0.1, grad=True),
        # one token between two blocks of a decoder
        dict(name="norm_decode", op="norm", T=1, H=2048, dtype="bf16", pad=0, gate="token", next=True, alpha=1.0),
        # the expert block's learner batch, forward
        dict(name="norm_learner", op="norm", T=32768, H=2048, dtype="bf16", pad=0, gate="token", next=True, alpha=0.5),
        # the same, backward
        dict(name="norm_learner_backward", op="norm_backward", T=32768, H=2048, dtype="bf16", pad=0, gate="token",
             next=True, alpha=0.5),
        # an odd width in float32, one gate row for each of seven sequences, backward
        dict(name="norm_odd_backward", op="norm_backward", T=777, H=1001, dtype="f32", pad=3, gate="sequence",
             next=False, alpha=1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_backward", "distill", "distill", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    pad = rng.choice([0, 0, 0, 8, rng.randint(1, 64)])
    if op.startswith("norm"):
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        T = _log_int(rng, 1, max(1, min(32768, (1 << 26) // H)))
        gate = rng.choice(["none", "token", "sequence"])
        if gate == "sequence":
            T = max(7, T // 7 * 7)
        return dict(op=op, T=T, H=H, dtype=dtype, pad=pad, gate=gate, next=rng.random() < 0.6,
                    alpha=rng.choice([1.0, 0.5, 1.25]))
    V = _log_int(rng, 1000, 262144)
    if rng.random() < 0.5:
        V = V // 64 * 64
    T = _log_int(rng, 1, max(1, min(8192, (1 << 30) // (V * (2 if dtype == "f32" else 1)))))
    case = dict(op=op, T=T, V=V, dtype=dtype, pad=pad, scale=rng.choice([1.0, 1.0, 0.8, 1.4]),
                masked=rng.choice([0.0, 0.0, 0.3, 0.9]))
    if op == "logprobs":
        T = min(T, max(1, (1 << 28) // V))
        case.update(T=T, ignored=rng.choice([0.0, 0.2]), top_k=rng.choice([0, 1, 5, 20, _log_int(rng, 2, 128)]))
    elif op == "logprobs_backward":
        case.update(ignored=rng.choice([0.0, 0.2]), entropy=rng.random() < 0.5)
    else:
        case.update(K=_log_int(rng, 1, 128), tail=rng.random() < 0.5, short=rng.choice([0.0, 0.3]),
                    grad=rng.random() < 0.6)
    return case


# ------------------------------------------------------------------------------- inputs

def _logits(case, gen):
    """Rows like a language model's: a broad background and, in every row, 48 tokens that
    stand out; a share of the vocabulary excluded (-inf) where the case has a mask.  Returns
    the logits (a view of padded storage) and 128 ids of each row that are never excluded,
    the 48 first."""
    T, V = case["T"], case["V"]
    store = torch.empty(T, V + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")
    # 128 places, distinct within a row; the first 48 stand out
    i = torch.arange(128, device="cuda")
    ids = (torch.randint(0, V, (T, 1), generator=gen, device="cuda") + (i % 48) * (V // 48) + i // 48) % V
    boost = (3.0 + 9.0 * torch.rand(T, 128, generator=gen, device="cuda") ** 2) * (i < 48)
    step = max(1, (1 << 27) // V)
    for a in range(0, T, step):
        b = min(T, a + step)
        z = torch.randn(b - a, V + case["pad"], generator=gen, device="cuda").mul_(2.0)
        if case["masked"] > 0.0:
            drop = torch.rand(b - a, V + case["pad"], generator=gen, device="cuda") < case["masked"]
            z.masked_fill_(drop, float("-inf"))
        best = torch.randn(b - a, 128, generator=gen, device="cuda").add_(boost[a:b])
        z.scatter_(1, ids[a:b], best)
        store[a:b] = z.to(store.dtype)
    return store[:, :V], ids


def _targets(case, ids, gen):
    T = case["T"]
    pick = torch.randint(0, 48, (T, 1), generator=gen, device="cuda")
    y = ids.gather(1, pick).squeeze(1)
    skip = torch.rand(T, generator=gen, device="cuda") < case["ignored"]
    return torch.where(skip, torch.full_like(y, IGNORE), y).to(torch.int32)


def _loss_scale(case):
    """Half-precision gradients travel with a loss scale."""
    return 1024.0 if case["dtype"] == "f16" else 1.0


def _teacher(case, ids, gen):
    """A teacher's list of every row: K distinct ids, best first, with the log
    probabilities of its own logits; short lists end in empty places (id -1)."""
    T, K = case["T"], case["K"]
    t = torch.randn(T, K, generator=gen, device="cuda") * 2.0
    t[:, :48] += 4.0
    t, order = t.sort(dim=1, descending=True)
    cand = ids[:, :K].gather(1, order)
    mass = 0.5 + 0.49 * torch.rand(T, 1, generator=gen, device="cuda")
    t = t - t.logsumexp(1, keepdim=True) + mass.log()
    if case["short"] > 0.0:
        keep = torch.where(torch.rand(T, 1, generator=gen, device="cuda") < case["short"],
                           torch.randint(0, K + 1, (T, 1), generator=gen, device="cuda"),
                           torch.full((T, 1), K, device="cuda"))
        cand = torch.where(torch.arange(K, device="cuda")[None, :] < keep, cand, torch.full_like(cand, -1))
    return cand.to(torch.int32).contiguous(), t.to(torch.float32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case=case)
    op = case["op"]
    if op.startswith("norm"):
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]

        def act(std=1.0):
            return (torch.randn(T, H + case["pad"], generator=gen, device="cuda") * std).to(dt)[:, :H]

        state["weight"] = 1.0 + 0.2 * torch.randn(H, generator=gen, device="cuda")
        state["next_weight"] = 1.0 + 0.2 * torch.randn(H, generator=gen, device="cuda") if case["next"] else None
        if case["gate"] == "token":
            state["gate"] = torch.rand(T, generator=gen, device="cuda")
        elif case["gate"] == "sequence":
            state["gate"] = torch.randn(7, H, generator=gen, device="cuda")
        else:
            state["gate"] = None
        state["x"], state["y"] = act(2.0), act(0.3)
        if op == "norm_backward":
            # what the forward leaves behind, and the gradients that arrive
            r, _, rstd_y, rstd_r = _norm_plain(state)
            state.update(r=r, rstd_y=rstd_y, rstd_r=rstd_r, dr=act(), dn=act() if case["next"] else None)
        return state
    z, ids = _logits(case, gen)
    state["logits"] = z
    if op == "distill":
        state["ids"], state["values"] = _teacher(case, ids, gen)
        state["dloss"] = torch.full((case["T"],), _loss_scale(case) / case["T"], device="cuda")
        return state
    state["targets"] = _targets(case, ids, gen)
    if op == "logprobs_backward":
        T = case["T"]
        unit = _loss_scale(case) / math.sqrt(T)
        state["dlogprob"] = torch.randn(T, generator=gen, device="cuda") * unit
        state["dentropy"] = torch.full((T,), -0.01 * unit, device="cuda") if case["entropy"] else None
        lse = torch.empty(T, device="cuda")
        ent = torch.empty(T, device="cuda")
        for a, b in _rows(case):
            _, lse[a:b], ent[a:b] = _stats_plain(z[a:b], state["targets"][a:b], case["scale"])
        state["lse"], state["entropy"] = lse, ent if case["entropy"] else None
    return state


# ------------------------------------------------------------------------------- plain forms

def _rows(case):
    step = max(1, (1 << 28) // case["V"])
    return [(a, min(case["T"], a + step)) for a in range(0, case["T"], step)]


def _stats_plain(z, targets, scale):
    """logprob, lse and entropy of rows of logits, float32."""
    c = z.float() * scale
    skip = targets == IGNORE
    m = c.amax(1, keepdim=True)
    lse = (c - m).exp().sum(1).log() + m.squeeze(1)
    lp = c - lse[:, None]
    logprob = lp.gather(1, targets.clamp(min=0).long()[:, None]).squeeze(1)
    p = lp.exp()
    entropy = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    zero = torch.zeros_like(lse)
    return torch.where(skip, zero, logprob), torch.where(skip, zero, lse), torch.where(skip, zero, entropy)


def _top_plain(z, lse, targets, scale, k):
    """The k best (value, then lowest id), by one whole-number key per token."""
    V = z.shape[1]
    f = z.float()
    bits = f.view(torch.int32).long()
    bits = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits)      # order of the values
    bits = torch.where(f == 0, torch.zeros_like(bits), bits)          # the two zeros are one value
    key = bits * (1 << 20) + (V - 1 - torch.arange(V, device=z.device))
    ids = key.topk(k, dim=1).indices
    val = f.gather(1, ids)
    lp = val * scale - lse[:, None]
    none = (val == float("-inf")) | (targets == IGNORE)[:, None]
    return (torch.where(none, torch.full_like(lp, float("-inf")), lp),
            torch.where(none, torch.full_like(ids, -1), ids).to(torch.int32))


def _logprobs_plain(state):
    case, z, y = state["case"], state["logits"], state["targets"]
    outs = []
    for a, b in _rows(case):
        one = list(_stats_plain(z[a:b], y[a:b], case["scale"]))
        if case["top_k"]:
            one += _top_plain(z[a:b], one[1], y[a:b], case["scale"], case["top_k"])
        outs.append(one)
    return [torch.cat(o) for o in zip(*outs)]


def _logprobs_backward_plain(state):
    case, z, y = state["case"], state["logits"], state["targets"]
    out = torch.empty(z.shape, dtype=z.dtype, device=z.device)
    for a, b in _rows(case):
        c = z[a:b].float() * case["scale"]
        lp = c - state["lse"][a:b, None]
        p = lp.exp()
        skip = y[a:b] == IGNORE
        g = state["dlogprob"][a:b, None]
        d = -g * p
        hit = torch.zeros_like(d).scatter_(1, y[a:b].clamp(min=0).long()[:, None], 1.0)
        d = d + g * hit
        if state["dentropy"] is not None:
            d = d - state["dentropy"][a:b, None] * p * (lp + state["entropy"][a:b, None])
        d = torch.where(torch.isinf(c) | skip[:, None], torch.zeros_like(d), d)
        out[a:b] = (d * case["scale"]).to(z.dtype)
    return out


def _distill_plain(state):
    case, z = state["case"], state["logits"]
    out = torch.empty(z.shape, dtype=z.dtype, device=z.device) if case["grad"] else None
    losses, lses = [], []
    for a, b in _rows(case):
        c = z[a:b].float() * case["scale"]
        ids, t = state["ids"][a:b].long(), state["values"][a:b]
        live = ids >= 0
        none = ~live.any(1)
        t = torch.where(live, t, torch.full_like(t, float("-inf")))
        if case["tail"]:
            q = t.exp()
        else:
            e = (t - t.amax(1, keepdim=True)).exp()
            q = e / e.sum(1, keepdim=True)
        q = torch.where(live, q, torch.zeros_like(q))
        lq = torch.where(q > 0, q.log(), torch.zeros_like(q))
        m = c.amax(1, keepdim=True)
        lse = (c - m).exp().sum(1, keepdim=True).log() + m
        lp = c - lse
        at = lp.gather(1, ids.clamp(min=0))
        loss = torch.where(q > 0, q * (lq - at), torch.zeros_like(q)).sum(1)
        if case["tail"]:
            # the mass outside the list, summed on its own
            inside = torch.zeros_like(c, dtype=torch.bool)
            row, col = live.nonzero(as_tuple=True)
            inside[row, ids[row, col]] = True
            rest = torch.where(inside, torch.full_like(c, float("-inf")), c)
            mr = rest.amax(1, keepdim=True)
            lr = ((rest - mr).exp().sum(1, keepdim=True).log() + mr - lse).squeeze(1)
            qr = (1.0 - q.sum(1)).clamp(min=0.0)
            use = (qr > 0) & ~torch.isnan(lr) & ~torch.isinf(lr)
            loss = loss + torch.where(use, qr * (qr.log() - lr), torch.zeros_like(qr))
        losses.append(torch.where(none, torch.zeros_like(loss), loss))
        lses.append(torch.where(none, torch.zeros_like(loss), lse.squeeze(1)))
        if out is not None:
            w = state["dloss"][a:b, None] * case["scale"]
            p = lp.exp()
            if case["tail"]:
                cut = torch.where(use, qr / lr.exp(), torch.zeros_like(qr))
                p = torch.where(inside, p, p * (1.0 - cut[:, None]))
            d = p.scatter_add(1, ids.clamp(min=0), -q)
            d = torch.where(torch.isinf(c) | none[:, None], torch.zeros_like(d), d * w)
            out[a:b] = d.to(z.dtype)
    return [torch.cat(losses), torch.cat(lses) if out is None else out]


def _gate_rows(gate, T):
    if gate is None:
        return 1.0
    return gate[:, None] if gate.dim() == 1 else gate.repeat_interleave(T // gate.shape[0], 0)


def _norm_plain(state):
    case = state["case"]
    dt = state["x"].dtype
    x, y = state["x"].float(), state["y"].float()
    rstd_y = torch.rsqrt((y * y).mean(1) + EPS)
    r = case["alpha"] * x + _gate_rows(state["gate"], x.shape[0]) * (y * rstd_y[:, None] * state["weight"])
    r = r.to(dt)
    if not case["next"]:
        return r, None, rstd_y, None
    f = r.float()
    rstd_r = torch.rsqrt((f * f).mean(1) + EPS)
    return r, (f * rstd_r[:, None] * state["next_weight"]).to(dt), rstd_y, rstd_r


def _norm_backward_plain(state):
    case, dt, T = state["case"], state["y"].dtype, state["y"].shape[0]
    d = state["dr"].float()
    out = []
    if case["next"]:
        rhat = state["r"].float() * state["rstd_r"][:, None]
        dn = state["dn"].float()
        u = dn * state["next_weight"]
        d = d + state["rstd_r"][:, None] * (u - rhat * (u * rhat).mean(1, keepdim=True))
        out = [(dn * rhat).sum(0)]
    gate = _gate_rows(state["gate"], T)
    yhat = state["y"].float() * state["rstd_y"][:, None]
    u = d * gate * state["weight"]
    dy = state["rstd_y"][:, None] * (u - yhat * (u * yhat).mean(1, keepdim=True))
    dweight = (d * gate * yhat).sum(0)
    dgate = []
    if state["gate"] is not None:
        full = d * state["weight"] * yhat
        G = state["gate"].shape[0]
        dgate = [full.sum(1) if state["gate"].dim() == 1 else full.view(G, T // G, -1).sum(1)]
    return [(case["alpha"] * d).to(dt), dy.to(dt), dweight] + dgate + out


# ------------------------------------------------------------------------------- one pass

def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        import nvfp4_w4a4_moe_quantize_gb300 as lib
        if op == "logprobs":
            out = lib.token_logprobs(state["logits"], state["targets"], top_k=case["top_k"], scale=case["scale"],
                                     ignore_index=IGNORE)
        elif op == "logprobs_backward":
            return lib.token_logprobs_backward(state["logits"], state["lse"], state["targets"], state["dlogprob"],
                                               entropy=state["entropy"], dentropy=state["dentropy"],
                                               scale=case["scale"], ignore_index=IGNORE)
        elif op == "distill":
            if case["grad"]:
                out = lib.distill_topk_backward(state["logits"], state["ids"], state["values"], state["dloss"],
                                                tail=case["tail"], scale=case["scale"])
            else:
                out = lib.distill_topk(state["logits"], state["ids"], state["values"], tail=case["tail"],
                                       scale=case["scale"])
        elif op == "norm":
            out = lib.moe_norm_out(state["x"], state["y"], state["weight"], gate=state["gate"],
                                   residual_scale=case["alpha"], next_weight=state["next_weight"], eps=EPS)
        else:
            out = lib.moe_norm_out_backward(state["dr"], state["y"], state["rstd_y"], state["weight"],
                                            gate=state["gate"], residual_scale=case["alpha"], dn=state["dn"],
                                            r=state["r"], rstd_r=state["rstd_r"], next_weight=state["next_weight"])
        return [o for o in out if o is not None]
    if op == "logprobs":
        return _logprobs_plain(state)
    if op == "logprobs_backward":
        return _logprobs_backward_plain(state)
    if op == "distill":
        return _distill_plain(state)
    if op == "norm":
        return [o for o in _norm_plain(state) if o is not None]
    return _norm_backward_plain(state)


def work(case):
    T, e, op = case["T"], BYTES[case["dtype"]], case["op"]
    if op.startswith("norm"):
        n = T * case["H"]
        gate = {"none": 0, "token": T, "sequence": 7 * case["H"]}[case["gate"]]
        if op == "norm":
            return {"bytes": n * e * (4 if case["next"] else 3) + 4 * gate + 8 * T,
                    "flops": n * (10 if case["next"] else 6)}
        return {"bytes": n * e * (6 if case["next"] else 4) + 8 * gate + 8 * T,
                "flops": n * (24 if case["next"] else 14)}
    n = T * case["V"]
    if op == "logprobs":
        return {"bytes": n * e + 16 * T + 8 * T * case["top_k"], "flops": 6 * n}
    if op == "logprobs_backward":
        return {"bytes": 2 * n * e + 20 * T, "flops": (7 if case["entropy"] else 4) * n}
    return {"bytes": n * e * (2 if case["grad"] else 1) + 8 * T * case["K"] + 8 * T,
            "flops": (8 if case["grad"] else 4) * n}


# ------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions in float64, row block by row block."""
    state = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op.startswith("norm"):
        return _exact_norm(case, state)
    z, s = state["logits"], case["scale"]
    if op == "logprobs":
        parts = [_exact_logprobs(case, z[a:a + 64].double() * s, z[a:a + 64], state["targets"][a:a + 64])
                 for a in range(0, T, 64)]
        return [torch.cat(p) for p in zip(*parts)]
    if op == "logprobs_backward":
        out = torch.empty(z.shape, dtype=torch.float64, device=z.device)
        for a in range(0, T, 64):
            b = min(T, a + 64)
            lp = torch.log_softmax(z[a:b].double() * s, 1)
            p = lp.exp()
            y = state["targets"][a:b].long()
            d = -p
            d[torch.arange(b - a, device=z.device), y.clamp(min=0)] += 1.0
            d *= state["dlogprob"][a:b, None].double()
            if case["entropy"]:
                plogp = torch.nan_to_num(p * lp, nan=0.0)
                d -= state["dentropy"][a:b, None].double() * (plogp - p * plogp.sum(1, keepdim=True))
            d[(y == IGNORE)[:, None] | (z[a:b] == float("-inf"))] = 0.0
            out[a:b] = d * s
        return out
    parts = [_exact_distill(case, z[a:a + 64].double() * s, state["ids"][a:a + 64].long(),
                            state["values"][a:a + 64].double(), state["dloss"][a:a + 64].double())
             for a in range(0, T, 64)]
    return [torch.cat(p) for p in zip(*parts)]


def _exact_logprobs(case, c, z, y):
    lp = torch.log_softmax(c, 1)
    skip = y == IGNORE
    lse = torch.logsumexp(c, 1)
    entropy = -torch.nan_to_num(lp.exp() * lp, nan=0.0).sum(1)
    at = lp.gather(1, y.clamp(min=0).long()[:, None]).squeeze(1)
    out = [v.masked_fill(skip, 0.0) for v in (at, lse, entropy)]
    if case["top_k"]:
        # a stable sort keeps equal values in the order of their ids
        order = z.float().sort(dim=1, descending=True, stable=True).indices[:, :case["top_k"]]
        val = lp.gather(1, order)
        none = torch.isinf(val) | skip[:, None]
        out += [val.masked_fill(none, float("-inf")), order.masked_fill(none, -1).to(torch.int32)]
    return out


def _exact_distill(case, c, ids, t, w):
    n, V = c.shape
    live = ids >= 0
    lp = torch.log_softmax(c, 1)
    q = t.exp() * live
    if not case["tail"]:
        q = torch.nan_to_num(q / q.sum(1, keepdim=True), nan=0.0)
    teacher = torch.zeros(n, V + 1, dtype=torch.float64, device=c.device)
    teacher.scatter_add_(1, torch.where(live, ids, torch.full_like(ids, V)), q)
    teacher = teacher[:, :V]
    listed_ = torch.zeros(n, V + 1, dtype=torch.float64, device=c.device)
    listed_.scatter_(1, torch.where(live, ids, torch.full_like(ids, V)), 1.0)
    listed_ = listed_[:, :V] > 0
    some = live.any(1)
    loss = torch.nan_to_num(torch.xlogy(teacher, teacher) - teacher * lp, nan=0.0).sum(1)
    grad = lp.exp() - teacher
    if case["tail"]:
        rest = torch.logsumexp(lp.masked_fill(listed_, float("-inf")), 1)
        qr = (1.0 - q.sum(1)).clamp(min=0.0)
        use = (qr > 0) & torch.isfinite(rest)
        loss = loss + torch.where(use, torch.xlogy(qr, qr) - qr * rest, torch.zeros_like(qr))
        cut = torch.where(use, qr / rest.exp(), torch.zeros_like(qr))
        grad = torch.where(listed_, grad, lp.exp() * (1.0 - cut)[:, None])
    loss = loss * some
    if not case["grad"]:
        return [loss, torch.logsumexp(c, 1) * some]
    grad = grad * (w * some)[:, None] * case["scale"]
    return [loss, grad.masked_fill(torch.isinf(c), 0.0)]


def _exact_norm(case, state):
    T, H = case["T"], case["H"]
    y, w = state["y"].double(), state["weight"].double()
    gate = state["gate"]
    if gate is None:
        g = torch.ones(T, 1, dtype=torch.float64, device=y.device)
    elif gate.dim() == 1:
        g = gate.double().reshape(T, 1)
    else:
        g = gate.double()[torch.arange(T, device=y.device) // (T // gate.shape[0])]
    if case["op"] == "norm":
        ry = 1.0 / torch.sqrt(y.square().sum(1) / H + EPS)
        r = case["alpha"] * state["x"].double() + g * y * ry[:, None] * w
        if not case["next"]:
            return [r, ry]
        # the second norm reads r as it is stored
        f = r.to(state["x"].dtype).double()
        rr = 1.0 / torch.sqrt(f.square().sum(1) / H + EPS)
        return [r, f * rr[:, None] * state["next_weight"].double(), ry, rr]
    d = state["dr"].double()
    out = []
    if case["next"]:
        r, rr, dn = state["r"].double(), state["rstd_r"].double()[:, None], state["dn"].double()
        v = dn * state["next_weight"].double()
        d = d + rr * v - r * rr ** 3 * ((v * r).sum(1, keepdim=True) / H)
        out = [(dn * r * rr).sum(0)]
    ry = state["rstd_y"].double()[:, None]
    v = d * g * w
    dy = ry * v - y * ry ** 3 * ((v * y).sum(1, keepdim=True) / H)
    res = [case["alpha"] * d, dy, (d * g * y * ry).sum(0)]
    if gate is not None:
        e = d * w * y * ry
        res.append(e.sum(1) if gate.dim() == 1 else e.reshape(gate.shape[0], -1, H).sum(1))
    return res + out
