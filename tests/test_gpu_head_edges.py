"""Log probabilities from hidden rows and the head's weight at the ends of their range."""
import numpy as np
import pytest
import torch

from oracle import ends as O
from test_gpu_head import HALF_STEP, IGNORE, U, f64, head, softmax_bound, store

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 140, 200, 300])
@pytest.mark.parametrize("far", [-3.3895e38, -1e37, -3e36])
def test_groups_of_tokens_far_below_the_rest(cuda_lib, T, far):
    """A padded vocabulary, switched off by a bias column at BF16's lowest value: whole groups of 128 tokens whose
    logits are finite and far off.  Everything is as without them."""
    V, H = 300, 40
    rng = np.random.default_rng(T)
    x, w = rng.integers(-2, 3, (T, H)).astype(float), rng.integers(-2, 3, (640, H)) / 32.0
    x[:, 0], w[:, 0], w[V:, 0] = 1.0, 0.0, far
    xt, wt = store(x, "bf16"), store(w, "bf16")
    y = rng.integers(0, V, T).astype(np.int32)
    y[1] = IGNORE
    yt = torch.from_numpy(y).cuda()
    lp, lse, ent = cuda_lib.head_logprobs(xt, wt, yt)
    want = O.head_logprobs(x, w[:V], y)
    # whole numbers over 32: the logits are exact, the softmax's bound is left
    tol = softmax_bound(x @ w[:V].T) + 4 * U * (1 + np.abs(want["lse"]))
    assert np.all(np.abs(f64(lse) - want["lse"]) <= tol)
    assert np.all(np.abs(f64(lp) - want["logprob"]) <= 2 * tol + 4 * U * np.abs(want["logprob"]))
    assert np.all(np.abs(f64(ent) - want["entropy"]) <= 2 * tol * (2 + want["entropy"] + np.log(V)))
    g = torch.from_numpy(rng.normal(size=T)).float().cuda()
    h = torch.from_numpy(rng.normal(size=T)).float().cuda()
    dx, dw = cuda_lib.head_logprobs_backward(xt, wt, lse, yt, g, ent, h)
    near = cuda_lib.head_logprobs(xt, wt[:V], yt)
    # (a group that the vocabulary's end cuts sums its entropy in another order)
    assert torch.equal(lp, near[0]) and torch.equal(lse, near[1])
    nx, nw = cuda_lib.head_logprobs_backward(xt, wt[:V], lse, yt, g, ent, h)
    assert torch.equal(dw[:V], nw) and (dw[V:] == 0).all()
    # (dhidden may be cut into other parts: two roundings of the result, and its float32 sums')
    assert torch.isfinite(dx).all()
    assert ((dx - nx).float().abs() <= 2 * HALF_STEP["bf16"] * nx.float().abs() + 2.0 ** -18 * g.abs().max()).all()
    assert cuda_lib.nvfp4_status_check() == 0


@pytest.mark.parametrize("T", [3, 200, 300])
def test_one_token_far_above_the_rest(cuda_lib, T):
    """A single huge logit, and a large scale: the entropy is 0 and the gradients vanish, none is NaN."""
    V, H = 700, 16
    rng = np.random.default_rng(T)
    for dtype, top, scale in (("bf16", 2.0 ** 126, 1.0), ("f16", 2.0 ** 15, 2.0 ** 108)):
        x, w = np.zeros((T, H)), rng.integers(-2, 3, (V, H)).astype(float)
        x[:, 0] = 1.0
        w[:, 0] = rng.integers(-4, 4, V)
        w[333, 0] = top
        xt, wt = store(x, dtype), store(w, dtype)
        yt = torch.full((T,), 333, dtype=torch.int32, device="cuda")
        lp, lse, ent = cuda_lib.head_logprobs(xt, wt, yt, scale=scale)
        assert (lp == 0).all() and (ent == 0).all() and (lse == top * scale).all()
        one = torch.ones(T, device="cuda")
        dx, dw = cuda_lib.head_logprobs_backward(xt, wt, lse, yt, None, ent, one)
        assert (dx == 0).all() and (dw == 0).all()
    assert cuda_lib.nvfp4_status_check() == 0


def test_a_workspace_may_begin_at_any_16_bytes(cuda_lib):
    """Workspaces of just the asked size that begin 16 bytes behind a whole line: the same bits, nothing written
    around them."""
    for T, V, H, dtype in ((5, 300, 72, "bf16"), (100, 700, 136, "f16"), (300, 1000, 264, "bf16")):
        xt, wt, y, yt, rng = head(T, V, H, dtype, T)
        g = torch.from_numpy(rng.normal(size=T)).float().cuda()
        h = torch.from_numpy(0.1 * rng.normal(size=T)).float().cuda()
        lp, lse, ent = want = cuda_lib.head_logprobs(xt, wt, yt)
        want_d = cuda_lib.head_logprobs_backward(xt, wt, lse, yt, g, ent, h)
        for lead in (16, 48, 240):
            for op, call, wanted in (
                    (cuda_lib.OP_HEAD_LOGPROBS, lambda ws: cuda_lib.head_logprobs(xt, wt, yt, workspace=ws), want),
                    (cuda_lib.OP_HEAD_LOGPROBS_BACKWARD,
                     lambda ws: cuda_lib.head_logprobs_backward(xt, wt, lse, yt, g, ent, h, workspace=ws), want_d)):
                n = cuda_lib.load().nvfp4_workspace_size(op, T, V, 0, H, 0)
                buf = torch.full((lead + n + 256,), 0x5A, dtype=torch.uint8, device="cuda")
                assert buf.data_ptr() % 256 == 0
                got = call(buf[lead:lead + n])
                assert all(torch.equal(a, b) for a, b in zip(got, wanted))
                assert (buf[:lead] == 0x5A).all() and (buf[lead + n:] == 0x5A).all()
    assert cuda_lib.nvfp4_status_check() == 0


def test_a_workspace_for_the_largest_batch_serves_the_smaller_ones(cuda_lib):
    V, H = 9000, 72
    ws = [torch.empty(cuda_lib.load().nvfp4_workspace_size(op, 700, V, 0, H, 0), dtype=torch.uint8, device="cuda")
          for op in (cuda_lib.OP_HEAD_LOGPROBS, cuda_lib.OP_HEAD_LOGPROBS_BACKWARD)]
    for T in (700, 1, 32, 33, 64, 65, 128, 129, 257, 600):
        xt, wt, y, yt, rng = head(T, V, H, "f16", T)
        g = torch.from_numpy(rng.normal(size=T)).float().cuda()
        want = cuda_lib.head_logprobs(xt, wt, yt)
        want_d = cuda_lib.head_logprobs_backward(xt, wt, want[1], yt, g)
        got = cuda_lib.head_logprobs(xt, wt, yt, workspace=ws[0])
        got_d = cuda_lib.head_logprobs_backward(xt, wt, want[1], yt, g, workspace=ws[1])
        assert all(torch.equal(a, b) for a, b in zip((*got, *got_d), (*want, *want_d))), T
    z = torch.randn(5000, 16, device="cuda")
    ids = torch.zeros(5000, 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(cuda_lib.load().nvfp4_workspace_size(cuda_lib.OP_BALANCE_LOSS, 5000, 1, 16, 0, 0), dtype=torch.uint8,
                     device="cuda")
    for T in (5000, 4864, 4865, 300, 7):
        want, got = cuda_lib.moe_balance_loss(z[:T], ids[:T]), cuda_lib.moe_balance_loss(z[:T], ids[:T], workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), T
    assert cuda_lib.nvfp4_status_check() == 0


@pytest.mark.parametrize("T,H,same", [(65, 264, False), (128, 72, False), (129, 264, False), (300, 1032, False),
                                      (1100, 328, False), (700, 136, True), (33000, 64, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_targets_part_of_d_is_not_rounded_twice(cuda_lib, T, H, same, dtype):
    """Targets that no row expects: d is -dlogprob there, any float32, and what it adds shows the result's own
    rounding alone.  The other tokens have no weight in the columns that are looked at."""
    V, common = 631, 400
    rng = np.random.default_rng(T)
    w = np.zeros((V, H))
    w[:common, 1:8] = rng.normal(0, 0.2, (common, 7))
    w[common:, 0], w[common:, 8:] = -40.0, rng.choice([-1, 1], (V - common, H - 8)) * rng.uniform(0.02, 0.04, (V - common, H - 8))
    x = rng.normal(size=(T, H))
    x[:, 0] = 1.0
    xt, wt = store(x, dtype), store(w, dtype)
    y = np.full(T, V - 1, np.int32) if same else rng.integers(common, V, T).astype(np.int32)
    y[rng.random(T) < 0.1] = IGNORE
    g = rng.uniform(0.5, 2.0, T) * np.where(same, 1.0, rng.choice([-1, 1], T))
    yt, gt = torch.from_numpy(y).cuda(), torch.from_numpy(g).float().cuda()
    _, lse, _ = cuda_lib.head_logprobs(xt, wt, yt, entropy=False)
    dx, dw = cuda_lib.head_logprobs_backward(xt, wt, lse, yt, gt)
    on = y != IGNORE
    g, x, w = f64(gt) * on, f64(xt), f64(wt)
    hit = np.zeros((T, V - common))
    hit[np.arange(T)[on], y[on] - common] = g[on]
    # (p of the targets is below e^-25; float32 sums of up to T addends, cut off towards zero 2.4 units a step of 16)
    tiny = 2.0 ** -20 + (T / 16) * 2.0 ** -22
    all_x, all_w = (np.abs(g)[:, None] * np.abs(x)).sum(0), np.abs(g)[:, None] * np.abs(w[common:, 8:]).sum(0)
    for got, want, mag, most in ((f64(dx)[:, 8:], hit @ w[common:, 8:], np.abs(hit) @ np.abs(w[common:, 8:]), all_w),
                                 (f64(dw)[common:], hit.T @ x, np.abs(hit).T @ np.abs(x), all_x)):
        tol = HALF_STEP[dtype] * np.abs(want) + tiny * mag + 2.0 ** -36 * most + (2.0 ** -24 if dtype == "f16" else 0.0)
        bad = np.abs(got - want) > tol
        assert not bad.any(), (bad.mean(), got[bad][:4], want[bad][:4])
    again = cuda_lib.head_logprobs_backward(xt, wt, lse, yt, gt)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    assert cuda_lib.nvfp4_status_check() == 0


def slope(got, want):
    """The mean relative error, weighted by want^2: what roundings of either sign leave out, and a cut does not."""
    return ((got.double() - want) * want).sum().item() / (want * want).sum().item()


def test_long_sums_of_the_hidden_rows_gradient(cuda_lib):
    """dhidden of rows whose target comes first among 131072 tokens: w_y is added at the start, and every later
    step cuts the sum off.  In a single sum of 8192 steps that takes 3e-4 of the result."""
    T, V, H = 2048, 131072, 1280
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(V, H, generator=gen, device="cuda").half()
    x = (torch.randn(T, H, generator=gen, device="cuda") * 0.01).half()
    y = torch.randint(0, 64, (T,), generator=gen, device="cuda", dtype=torch.int32)
    g = torch.ones(T, device="cuda")
    _, lse, _ = cuda_lib.head_logprobs(x, w, y, entropy=False)
    dx, _ = cuda_lib.head_logprobs_backward(x, w, lse, y, g, need_weight=False)
    want, wd = torch.empty(T, H, dtype=torch.float64, device="cuda"), w.double()
    for a in range(0, T, 256):
        d = -torch.softmax(x[a:a + 256].double() @ wd.t(), 1)
        d.scatter_add_(1, y[a:a + 256].long()[:, None], torch.ones(256, 1, dtype=torch.float64, device="cuda"))
        want[a:a + 256] = d @ wd
    # 512 steps a stretch of at most 2^-23 of a sum that is w_y up to some percent (half of it on average: the small
    # addends' own cuts are of either sign); d_y = 1 - p_y, p_y about 2^-17, is rounded to 1; 2^-16 for the other
    # roundings, of either sign and of 2.6 million elements (2^-11 / 1000 for each kind)
    assert abs(slope(dx, want)) <= 512 * 2.0 ** -23 * 1.1 + 2.0 ** -16 + 2.0 ** -16
    assert cuda_lib.nvfp4_status_check() == 0


def test_long_sums_of_the_weights_gradient(cuda_lib):
    """dweight of 262144 rows, of which the first 64 weigh 4096 times as much as the others."""
    T, V, H = 262144, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = (torch.randn(V, H, generator=gen, device="cuda") * 0.05).half()
    x = torch.randn(T, H, generator=gen, device="cuda").half()
    y = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    g = torch.full((T,), 2.0 ** -12, device="cuda")
    g[:64] = 1.0
    _, lse, _ = cuda_lib.head_logprobs(x, w, y, entropy=False)
    _, dw = cuda_lib.head_logprobs_backward(x, w, lse, y, g, need_hidden=False)
    xd = x.double()
    d = torch.softmax(xd @ w.double().t(), 1).neg_()
    d.scatter_add_(1, y.long()[:, None], torch.ones(T, 1, dtype=torch.float64, device="cuda"))
    want = (d * g.double()[:, None]).t() @ xd
    # 512 steps a stretch of at most 2^-23 of a sum that is the first rows' up to a few percent; and eight deviations of the
    # roundings, uniform within 2^-11 of the value: the result's, and those of the heavy rows' d
    norm = (want * want).sum()
    own = (want ** 4).sum().sqrt() / norm
    heavy = (d[:64] * (xd[:64] @ want.t())).norm() / norm
    assert abs(slope(dw, want)) <= 512 * 2.0 ** -23 * 1.1 + 8 * 2.0 ** -11 / 3 ** 0.5 * (own + heavy).item()
    assert cuda_lib.nvfp4_status_check() == 0


def cut_steps(x, w, stretch):
    """What sums of x_h w_h >= 0 lose at most, added 16 products at a time, in stretches.  A step aligns its addends
    to the largest's exponent, the sum's, and keeps two bits below the last place: each product loses less than a
    quarter of a unit in the sum's last place, the new sum less than a unit."""
    p = (x * w).reshape(-1, 16).sum(1)
    lost = 0.0
    for a in range(0, len(p), stretch // 16):
        s = np.cumsum(p[a:a + stretch // 16])
        lost += (5 * 2.0 ** (np.floor(np.log2(np.maximum(s, 1e-300))) - 23)).sum()
    return lost


def test_long_logits_of_the_gradients(cuda_lib):
    """Logits that are long sums of one sign: p is exp of them, and d of 64 equally likely tokens shows their
    error whole.  In a single sum of 1024 steps the logits, about 56, lose 6e-3."""
    T, V, H = 1000, 192, 16384
    rng = np.random.default_rng(3)
    x = store(rng.uniform(0.9, 1.1, (T, H)) * 0.0625, "f16")
    w = store(np.where(np.arange(V)[:, None] < 64, 0.055, 0.0) + np.zeros((V, H)), "f16")
    y = torch.full((T,), V - 1, dtype=torch.int32, device="cuda")
    lse = torch.logsumexp(x.double() @ w.double().t(), 1).float()
    _, dw = cuda_lib.head_logprobs_backward(x, w, lse, y, torch.ones(T, device="cuda"), need_hidden=False)
    want = -(torch.full((T, 64), 1 / 64, dtype=torch.float64, device="cuda")).t() @ x.double()
    # the logits' cuts in stretches of 512 products (row by row the same to 1%); lse's rounding, the exponent's
    # and ex2's; eight deviations of the roundings of d, one a row (all 64 tokens share it), and of the result
    c = 1.01 * cut_steps(f64(x)[0], f64(w)[0], 512)
    tol = c + 64 * U + 20 * U + 8 * HALF_STEP["f16"] / 3 ** 0.5 * (T ** -0.5 + H ** -0.5)
    assert c < 5e-4 and abs(slope(dw[:64], want)) <= tol
    assert cuda_lib.nvfp4_status_check() == 0


@pytest.mark.parametrize("T", [40, 100, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gradients_of_almost_certain_rows(cuda_lib, T, dtype):
    """1 - p of a target that has nearly all the probability comes out right only from the very logits that made
    lse.  Seen in the sum of d over the tokens, which is 0: a column of ones in the weight."""
    V, H = 1000, 2048
    rng = np.random.default_rng(T)
    w = rng.normal(0, 0.1, (V, H))
    w[:, 0] = 1.0
    y = rng.integers(0, V, T).astype(np.int32)
    x = 0.7 * w[y]                                       # the target's logit is 14, a sum of squares
    x[:, 0] = 0.0
    xt, wt, yt = store(x, dtype), store(w, dtype), torch.from_numpy(y).cuda()
    _, lse, _ = cuda_lib.head_logprobs(xt, wt, yt, entropy=False)
    dx, _ = cuda_lib.head_logprobs_backward(xt, wt, lse, yt, torch.ones(T, device="cuda"))
    c = f64(xt) @ f64(wt).T
    p = np.exp(c - f64(lse)[:, None])
    rest = 1 - p[np.arange(T), y]
    assert rest.max() < 0.01
    # each d's rounding, of |d| adding up to 2 (1 - p); p by the softmax's error on both ways, lse's rounding
    tol = 2 * HALF_STEP[dtype] * (rest + 1e-4) + 2 * softmax_bound(c) + 8 * U * (1 + np.abs(f64(lse)))
    assert np.all(np.abs(f64(dx)[:, 0]) <= tol)
    assert cuda_lib.nvfp4_status_check() == 0


@pytest.mark.parametrize("T", [1, 200])
def test_a_logit_is_summed_in_short_stretches(cuda_lib, T):
    """One token, whose lse is its logit: 1, and a little less than a last place of it at every further step of 16
    products, which a sum without an end loses every time."""
    H = 2048
    x, w = np.ones((T, H)), np.full((1, H), 0.984375 * 2.0 ** -27)
    w[0, 0], w[0, 1:16] = 1.0, 0.0
    _, lse, ent = cuda_lib.head_logprobs(store(x, "bf16"), store(w, "bf16"))
    want = (x @ w.T)[:, 0]
    # 31 further steps of the first 512 products lose it; the other stretches do not; four sums' roundings
    assert np.all(np.abs(f64(lse) - want) <= 31 * 0.984375 * 2.0 ** -23 + 4 * U)
    assert (ent == 0).all() and cuda_lib.nvfp4_status_check() == 0


@pytest.mark.parametrize("T", [40, 140, 300])
@pytest.mark.parametrize("light", [2.0 ** -6, 2.0 ** -14, 2.0 ** -18, 2.0 ** -22])
def test_half_precision_rows_far_lighter_than_the_heaviest(cuda_lib, T, light):
    """A row's own token, which the heavier rows have no share in: its weight's gradient is the light row's alone, a
    normal number, and as exact as any."""
    V, H = 400, 48
    rng = np.random.default_rng(T)
    x = rng.choice([-1, 1], (T, H)) * rng.uniform(1.0, 3.9, (T, H))
    x[:, 0], x[0, 0] = 3.0, -3.0
    w = rng.normal(0, 0.05, (V, H))
    w[:, 0] = 0.0
    w[7, 0] = -20.0                                      # 60 for row 0, -60 for the others
    xt, wt = store(x, "f16"), store(w, "f16")
    y = rng.integers(8, V, T).astype(np.int32)
    y[0] = 300                                           # row 0: token 7 is almost certain, and not its target
    g = np.full(T, 1024.0)
    g[0] *= light
    yt, gt = torch.from_numpy(y).cuda(), torch.from_numpy(g).float().cuda()
    _, lse, _ = cuda_lib.head_logprobs(xt, wt, yt, entropy=False)
    dx, dw = cuda_lib.head_logprobs_backward(xt, wt, lse, yt, gt)
    want = -g[0] * f64(xt)[0]                            # dweight of token 7: p = 1
    # d's rounding (p within 2^-16 of 1), the hidden row's, which is exact where its numbers stay normal, the result's
    assert np.all(np.abs(f64(dw)[7] - want) <= np.abs(want) * (2 * HALF_STEP["f16"] * (1 + 2.0 ** -10) + 2.0 ** -15))
    want = g[0] * (f64(wt)[300] - f64(wt)[7])            # and the light row's own gradient
    assert np.all(np.abs(f64(dx)[0] - want) <= np.abs(want) * (2 * HALF_STEP["f16"]) + g[0] * 20 * 2.0 ** -15)
    assert cuda_lib.nvfp4_status_check() == 0
