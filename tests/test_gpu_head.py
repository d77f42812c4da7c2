"""Log probabilities from hidden rows and the head's weight, and their gradients, against the float64 oracle.

Bounds, u = 2^-24.  A logit is a sum of H exact products that a tensor core adds 16 at a time, cut off (not
rounded) at every step: within delta = 2 (H / 16 + 4) 2 u S of its value, S = scale sum_h |x_h w_h| (the largest of
the row).  The softmax adds, for exponents of at most D in base 2, 1.4 D u for the exponent's two roundings, 4 u for
ex2 and a rounding for each addition on the way.  d is rounded to 16 bits (half a step h of the type; of up to
64 rows to two such numbers, h^2) and carries p's error; the products of d are cut off like the logits, over K / 16
steps, relative to the sum of magnitudes."""
import numpy as np
import pytest
import torch

from oracle import ends as O
from oracle import learner as OL

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
IGNORE = -100


def f64(t):
    return t.detach().cpu().double().numpy()


def store(a, dtype, pad=0):
    t = torch.zeros(a.shape[0], a.shape[1] + pad, dtype=DT[dtype], device="cuda")[:, :a.shape[1]]
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def head(T, V, H, dtype, seed, pad=0, ignored=0.25):
    rng = np.random.default_rng(seed)
    w = store(rng.normal(0, 2.0 / np.sqrt(H), (V, H)), dtype, pad)
    y = rng.integers(0, V, T).astype(np.int32)
    x = store(rng.normal(size=(T, H)) + rng.uniform(0, 2, (T, 1)) * f64(w)[y], dtype, pad)
    y[rng.random(T) < ignored] = IGNORE
    return x, w, y, torch.from_numpy(y).cuda(), rng


def logit_bound(x, w, scale):
    """delta of every row."""
    H = x.shape[1]
    S = scale * (np.abs(x) @ np.abs(w).T).max(1)
    return 2 * (H / 16 + 4) * 2 * U * S


def softmax_bound(c):
    """Relative error of a sum of exponentials beyond the logits' own: the exponents, ex2, the additions."""
    D = 1.45 * (c.max(1) - c.min(1))
    return 1.4 * D * U + 4 * U + (64 + c.shape[1] / 4096 + 64 + 8) * U


def check_forward(lib, xt, wt, y, yt, scale=1.0, entropy=True, exact=False, status=0, **kw):
    lp, lse, ent = lib.head_logprobs(xt, wt, yt, scale=scale, entropy=entropy, **kw)
    assert lib.nvfp4_status_check() == status
    x, w = f64(xt), f64(wt)
    c = scale * O.head_logits(x, w)
    want = O.head_logprobs(x, w, y, scale)
    delta = 0.0 if exact else logit_bound(x, w, scale)
    r = softmax_bound(c)
    skip = np.zeros(x.shape[0], bool) if y is None else y == IGNORE
    base = delta + r + 4 * U * (1 + np.abs(want["lse"]))
    tol = np.where(skip, 0.0, base)
    assert np.all(np.abs(f64(lse) - want["lse"]) <= tol)
    if y is not None:
        ok = (y >= 0) & (y < w.shape[0])
        at = np.abs(want["logprob"])
        assert np.all((np.abs(f64(lp) - want["logprob"]) <= np.where(skip, 0.0, 2 * base + 4 * U * at))[ok | skip])
        assert np.isnan(f64(lp)[~ok & ~skip]).all()
    if entropy:
        # sum of p (ln s - ln e): every p off by base, its logarithm too
        tol = np.where(skip, 0.0, 2 * base * (2 + want["entropy"] + np.log(w.shape[0])))
        assert np.all(np.abs(f64(ent) - want["entropy"]) <= tol)
    return lp, lse, ent


def check_backward(lib, xt, wt, y, yt, lse, ent, g=None, h=None, scale=1.0, dtype="bf16", status=0, **kw):
    gt = None if g is None else torch.from_numpy(g.astype(np.float32)).cuda()
    ht = None if h is None else torch.from_numpy(h.astype(np.float32)).cuda()
    dx, dw = lib.head_logprobs_backward(xt, wt, lse, yt, gt, ent if h is not None else None, ht, scale=scale, **kw)
    assert lib.nvfp4_status_check() == status
    x, w = f64(xt), f64(wt)
    T, V = x.shape[0], w.shape[0]
    g32 = None if g is None else g.astype(np.float32)
    h32 = None if h is None else h.astype(np.float32)
    want_x, want_w, d = O.head_logprobs_backward(x, w, y, g32, h32, scale)
    c = scale * O.head_logits(x, w)
    lnp, p, wlse = OL.softmax_stats(c)
    live = np.ones(T) if y is None else (y != IGNORE).astype(np.float64)
    mag = np.zeros_like(p)
    if g is not None:
        ok = (y >= 0) & (y < V)
        mag += np.abs(g32)[:, None] * p * ok[:, None]
        mag[np.arange(T)[ok], y[ok]] += np.abs(g32)[ok]
    weight = np.zeros(T) if g is None else np.abs(g32).astype(np.float64)
    if h is not None:
        entropy = -(p * lnp).sum(1)
        mag += np.abs(h32)[:, None] * p * (np.abs(lnp) + entropy[:, None] + 1)
        weight = weight + 16 * np.abs(h32)
    mag *= scale * live[:, None]
    # of p: the logits here and in lse, the exponent, ex2; of d: its factors and its rounding
    perr = 2 * logit_bound(x, w, scale) + softmax_bound(c) + 8 * U * (1 + np.abs(wlse)) + 3 * U * np.abs(c).max(1)
    # (up to 64 rows d is two numbers: the second one's half step of the first one's)
    rounding = HALF_STEP[dtype] ** 2 * 2 if T <= 64 else HALF_STEP[dtype] * (1 + 2.0 ** -7)
    each = mag * (rounding + 2 * perr[:, None] + 8 * U)
    aw, ax = np.abs(w), np.abs(x) * live[:, None]
    tol_x = each @ aw + 4 * U * (V / 16 + 40) * (mag @ aw) + HALF_STEP[dtype] * np.abs(want_x)
    tol_w = each.T @ ax + 4 * U * (T / 16 + 8) * (mag.T @ ax) + HALF_STEP[dtype] * np.abs(want_w)
    if dtype == "f16":
        # d / r (r up to twice the row's weight, times 2^14) and x r / max r below the type's normal values
        r = 2 * scale * weight * live
        tol_x += 2.0 ** -39 * r[:, None] * aw.sum(0) + 2.0 ** -25
        tol_w += 2.0 ** -39 * (r[:, None] * ax).sum(0) + 2.0 ** -25
        tol_w += 2.0 ** -25 * r.max() * (mag / np.maximum(r, 1e-300)[:, None] * 2).sum(0)[:, None]
    for got, want, tol in ((dx, want_x, tol_x), (dw, want_w, tol_w)):
        if got is not None:
            bad = np.abs(f64(got) - want) > tol + 1e-38
            assert not bad.any(), (np.argwhere(bad)[:5], f64(got)[bad][:5], want[bad][:5], tol[bad][:5])
    return dx, dw


@pytest.mark.parametrize("T,V,H", [(1, 1, 8), (1, 127, 64), (3, 128, 72), (64, 129, 8), (65, 1000, 256), (128, 257, 136),
                                   (129, 300, 520), (256, 5000, 64), (257, 513, 328), (300, 2049, 1096), (700, 3001, 192)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_against_the_oracle(cuda_lib, T, V, H, dtype):
    xt, wt, y, yt, rng = head(T, V, H, dtype, T + V, pad=8 if T % 2 else 0)
    scale = 0.8 if T % 2 else 1.3
    lp, lse, ent = check_forward(cuda_lib, xt, wt, y, yt, scale)
    g, h = rng.normal(size=T), 0.1 * rng.normal(size=T)
    check_backward(cuda_lib, xt, wt, y, yt, lse, ent, g, None, scale, dtype)
    check_backward(cuda_lib, xt, wt, y, yt, lse, ent, g, h, scale, dtype)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 48, 63, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_few_rows_gradients_show_their_own_rounding_alone(cuda_lib, T, dtype):
    """Confident rows, whose gradient hangs on the target's d: its 16-bit rounding does not show."""
    V, H = 900, 328
    xt, wt, y, yt, rng = head(T, V, H, dtype, 100 + T, ignored=0.0)
    xt.copy_(f64_to(xt, f64(xt) + 1.5 * f64(wt)[y]))
    lp, lse, ent = check_forward(cuda_lib, xt, wt, y, yt)
    for h in (None, 0.1 * rng.normal(size=T)):
        check_backward(cuda_lib, xt, wt, y, yt, lse, ent, rng.normal(size=T), h, 1.0, dtype)


def f64_to(like, a):
    return torch.from_numpy(a.astype(np.float32)).to(like.dtype).cuda()


@pytest.mark.parametrize("T", [5, 200, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_exact_logits(cuda_lib, T, dtype):
    """Whole-number operands: every partial sum of a logit is exact, whatever cuts it off, so the results are
    as near as the softmax alone allows, at every length of the contraction."""
    for H in (64, 1032, 2056, 4104):
        rng = np.random.default_rng(H)
        x = store(rng.integers(-2, 3, (T, H)), dtype)
        w = store(rng.integers(-1, 2, (700, H)), dtype)
        y = rng.integers(0, 700, T).astype(np.int32)
        check_forward(cuda_lib, x, w, y, torch.from_numpy(y).cuda(), 1 / 32, exact=True)


def test_a_large_vocabulary(cuda_lib):
    """2^20 tokens, the last one the target."""
    V = 1 << 20
    xt, wt, y, yt, rng = head(2, V, 8, "bf16", 1, ignored=0.0)
    y[0] = V - 1
    yt[0] = V - 1
    _, lse, ent = check_forward(cuda_lib, xt, wt, y, yt)
    check_backward(cuda_lib, xt, wt, y, yt, lse, ent, rng.normal(size=2))


def test_pieces_of_the_vocabulary(cuda_lib):
    """Enough rows that the backward takes the vocabulary in several pieces: against float64 products of the whole d."""
    T, V, H = 32900, 17000, 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    w = (0.4 * torch.randn(V, H, generator=gen, device="cuda")).bfloat16()
    y = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    y[::3] = IGNORE
    g = torch.randn(T, generator=gen, device="cuda")
    lp, lse, _ = cuda_lib.head_logprobs(x, w, y)
    dx, dw = cuda_lib.head_logprobs_backward(x, w, lse, y, g)
    want_x, want_w = torch.zeros(T, H, dtype=torch.float64, device="cuda"), torch.zeros(V, H, dtype=torch.float64, device="cuda")
    mag_x, mag_w = want_x.clone(), want_w.clone()
    wd = w.double()
    for a in range(0, T, 4096):
        s = slice(a, min(T, a + 4096))
        xd, n = x[s].double(), min(T, a + 4096) - a
        p = torch.softmax(xd @ wd.t(), 1)
        hit = torch.zeros_like(p).scatter_(1, y[s].clamp(min=0).long()[:, None], 1.0)
        gs = (g[s].double() * (y[s] != IGNORE))[:, None]
        want_x[s] = (gs * (hit - p)) @ wd
        mag_x[s] = (gs.abs() * (hit + p)) @ wd.abs()
        want_w += (gs * (hit - p)).t() @ xd
        mag_w += (gs.abs() * (hit + p)).t() @ xd.abs()
    # d's rounding and p's error (delta <= 2 (40/16 + 4) 2 u 40 and the softmax's), the products over 17000 / 16 and
    # 32900 / 16 steps, the result's rounding
    rel = HALF_STEP["bf16"] * (1 + 2.0 ** -6) + 4 * U * 40 * 14 + 400 * U
    for got, want, mag, K in ((dx, want_x, mag_x, V), (dw, want_w, mag_w, T)):
        tol = (rel + 4 * U * (K / 16 + 40)) * mag + HALF_STEP["bf16"] * want.abs() + 1e-30
        assert ((got.double() - want).abs() <= tol).all()
    assert cuda_lib.nvfp4_status_check() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [7, 200, 400])
def test_ignored_rows_may_hold_anything(cuda_lib, T, dtype):
    V, H = 600, 136
    xt, wt, y, yt, rng = head(T, V, H, dtype, T, ignored=0.4)
    y[-1] = IGNORE
    yt.copy_(torch.from_numpy(y))
    g = torch.from_numpy(rng.normal(size=T)).float().cuda()
    h = torch.from_numpy(0.1 * rng.normal(size=T)).float().cuda()
    skip = yt == IGNORE
    want = cuda_lib.head_logprobs(xt, wt, yt)
    want_d = cuda_lib.head_logprobs_backward(xt, wt, want[1], yt, g, want[2], h)
    x2 = xt.clone()
    x2[skip] = torch.tensor([float("nan"), float("inf")], dtype=xt.dtype, device="cuda").repeat(H // 2)
    g[skip], h[skip] = float("nan"), float("inf")
    lse, ent = want[1].clone(), want[2].clone()
    lse[skip], ent[skip] = float("nan"), float("-inf")
    got = cuda_lib.head_logprobs(x2, wt, yt)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and all((o[skip] == 0).all() for o in got)
    got_d = cuda_lib.head_logprobs_backward(x2, wt, lse, yt, g, ent, h)
    assert all(torch.equal(a, b) for a, b in zip(got_d, want_d)) and (got_d[0][skip] == 0).all()
    # nothing to score at all
    none = torch.full_like(yt, IGNORE)
    x2[:] = float("nan")
    assert all((o == 0).all() for o in cuda_lib.head_logprobs(x2, wt, none))
    assert all((o == 0).all() for o in cuda_lib.head_logprobs_backward(x2, wt, lse, none, g, ent, h))
    assert cuda_lib.nvfp4_status_check() == 0


def test_a_row_s_bits_do_not_depend_on_the_batch(cuda_lib):
    """Rows alone, in small and large batches, among ignored rows: the same log probabilities, bit for bit."""
    V, H = 5003, 1160
    xt, wt, y, yt, _ = head(600, V, H, "bf16", 4, ignored=0.0)
    want = cuda_lib.head_logprobs(xt, wt, yt)
    for rows in ([0], [599], list(range(100)), list(range(50, 179)), list(range(300)), list(range(3, 600, 2))):
        r = torch.tensor(rows, device="cuda")
        got = cuda_lib.head_logprobs(xt[r], wt, yt[r])
        assert all(torch.equal(a, b[r]) for a, b in zip(got, want)), len(rows)
    y2 = yt.clone()
    y2[1::3] = IGNORE
    got = cuda_lib.head_logprobs(xt, wt, y2)
    keep = y2 != IGNORE
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, want))
    lp, lse, none = cuda_lib.head_logprobs(xt, wt, yt, entropy=False)
    assert none is None and torch.equal(lp, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("T", [30, 400])
def test_targets_outside_the_vocabulary(cuda_lib, T):
    V, H = 300, 64
    xt, wt, y, yt, rng = head(T, V, H, "bf16", 5)
    bad = [0, 11, 29]
    y[bad] = [-1, V, 2 ** 31 - 1]
    yt.copy_(torch.from_numpy(y))
    S = cuda_lib.Status.DEVICE_STATUS
    lp, lse, ent = check_forward(cuda_lib, xt, wt, y, yt, status=S)
    # their log probability adds nothing to the gradients, their entropy does
    check_backward(cuda_lib, xt, wt, y, yt, lse, ent, rng.normal(size=T), 0.1 * rng.normal(size=T))


def test_what_is_not_asked_for(cuda_lib):
    xt, wt, y, yt, rng = head(150, 400, 72, "bf16", 6, ignored=0.2)
    lp, lse, ent = cuda_lib.head_logprobs(xt, wt)                      # no targets: every row counts
    assert lp is None
    check_forward(cuda_lib, xt, wt, None, None)
    g, h = rng.normal(size=150), 0.1 * rng.normal(size=150)
    check_backward(cuda_lib, xt, wt, None, None, lse, ent, None, h)     # the entropy alone
    lp, lse, ent = cuda_lib.head_logprobs(xt, wt, yt)
    dx, dw = check_backward(cuda_lib, xt, wt, y, yt, lse, ent, g, h)
    gt, ht = torch.from_numpy(g).float().cuda(), torch.from_numpy(h).float().cuda()
    one = cuda_lib.head_logprobs_backward(xt, wt, lse, yt, gt, ent, ht, need_weight=False)
    two = cuda_lib.head_logprobs_backward(xt, wt, lse, yt, gt, ent, ht, need_hidden=False)
    assert one[1] is None and two[0] is None and torch.equal(one[0], dx) and torch.equal(two[1], dw)
    e = torch.empty(0, 72, dtype=xt.dtype, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    assert [o.shape[0] for o in cuda_lib.head_logprobs(e, wt, i)] == [0, 0, 0]
    f = torch.empty(0, device="cuda")
    dx, dw = cuda_lib.head_logprobs_backward(e, wt, f, i, f)
    assert dx.shape == (0, 72) and (dw == 0).all()
    # a single token and rows that have no pitch of their own
    lp, lse, ent = cuda_lib.head_logprobs(xt[:1], wt[:1], torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert lp.item() == 0 and ent.item() == 0
    assert cuda_lib.nvfp4_status_check() == 0


def test_half_precision_with_small_and_uneven_weights(cuda_lib):
    """Gradients far below the type's smallest d, and rows whose weights differ by a million: the large rows'
    gradients keep their bits."""
    T, V, H = 140, 3000, 64
    xt, wt, y, yt, rng = head(T, V, H, "f16", 7, ignored=0.0)
    lp, lse, ent = cuda_lib.head_logprobs(xt, wt, yt)
    for small in (1e-3, 1e-6):
        g = rng.normal(size=T) * np.where(np.arange(T) % 2, small, 1.0)
        check_backward(cuda_lib, xt, wt, y, yt, lse, ent, g, None, 1.0, "f16")
    check_backward(cuda_lib, xt, wt, y, yt, lse, ent, np.zeros(T), None, 1.0, "f16")
    g = np.full(T, 6e4)                                                # near the type's largest
    check_backward(cuda_lib, xt, wt, y, yt, lse, ent, g / T, None, 1.0, "f16")


def test_not_a_number_stays_in_its_row(cuda_lib):
    T = 300
    xt, wt, y, yt, _ = head(T, 500, 64, "bf16", 8, ignored=0.0)
    xt[3, 5], xt[270, 0] = float("nan"), float("inf")
    for s in (slice(0, 20), slice(0, T)):
        lp, lse, ent = cuda_lib.head_logprobs(xt[s], wt, yt[s])
        bad = torch.isnan(lse)
        assert bad[3] and bad.sum() == (2 if s.stop == T else 1)
        assert torch.equal(torch.isnan(lp), bad) and torch.equal(torch.isnan(ent), bad)


def test_deterministic_on_streams_and_in_graphs(cuda_lib):
    """Twice the same bits; a given stream; a forward and backward captured together and replayed on new inputs,
    two graphs of one workspace one after the other."""
    T, V, H = 300, 2500, 264
    xt, wt, y, yt, rng = head(T, V, H, "bf16", 9)
    g = torch.from_numpy(rng.normal(size=T)).float().cuda()
    h = torch.from_numpy(0.1 * rng.normal(size=T)).float().cuda()
    n = max(cuda_lib.load().nvfp4_workspace_size(op, T, V, 0, H, 0)
            for op in (cuda_lib.OP_HEAD_LOGPROBS, cuda_lib.OP_HEAD_LOGPROBS_BACKWARD))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step(**kw):
        lp, lse, ent = cuda_lib.head_logprobs(xt, wt, yt, **kw)
        return lp, lse, ent, *cuda_lib.head_logprobs_backward(xt, wt, lse, yt, g, ent, h, **kw)

    want = [o.clone() for o in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for got in (step(workspace=ws), step(stream=side)):
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(workspace=ws)
        graphs.append((graph, out))
    x2, _, _, y2, _ = head(T, V, H, "bf16", 10, ignored=0.6)
    for x, t in ((xt.clone(), yt.clone()), (x2, y2)):
        xt.copy_(x)
        yt.copy_(t)
        want = [o.clone() for o in step()]
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert cuda_lib.nvfp4_status_check() == 0


def test_gradients_against_differences(cuda_lib):
    """The gradients along random directions against differences of the float64 loss."""
    T, V, H = 40, 900, 64
    xt, wt, y, yt, rng = head(T, V, H, "f16", 11)
    g, h = rng.normal(size=T), 0.1 * rng.normal(size=T)
    lp, lse, ent = cuda_lib.head_logprobs(xt, wt, yt)
    dx, dw = cuda_lib.head_logprobs_backward(xt, wt, lse, yt, torch.from_numpy(g).float().cuda(), ent,
                                             torch.from_numpy(h).float().cuda())
    x, w = f64(xt), f64(wt)

    def f(a, b):
        out = O.head_logprobs(a, b, y)
        return (out["logprob"] * g).sum() + (out["entropy"] * h).sum()

    for _ in range(3):
        vx, vw = rng.normal(size=x.shape), rng.normal(size=w.shape)
        want = (f(x + 1e-5 * vx, w) - f(x - 1e-5 * vx, w)) / 2e-5
        # every element within 2^-9 of the largest: 2^-11 for its own rounding and for d's, and what cancels
        assert abs(want - (f64(dx) * vx).sum()) < 2.0 ** -9 * np.abs(f64(dx) * vx).sum()
        want = (f(x, w + 1e-5 * vw) - f(x, w - 1e-5 * vw)) / 2e-5
        assert abs(want - (f64(dw) * vw).sum()) < 2.0 ** -9 * np.abs(f64(dw) * vw).sum()
