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
