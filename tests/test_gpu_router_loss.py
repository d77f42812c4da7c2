"""The router's balance loss, per-expert counts and the gradient of the router's logits against the float64
oracle.

Bounds, u = 2^-24 (a float32 rounding).  p = exp(z - max) / sum: the exponent in base 2, d = (z - max) log2(e),
is rounded twice, so exp is off by 0.7 |d| 2 u, ex2 itself by 2^-22; numerator and denominator share that bound,
the sum over E experts adds E / 32 + 5 roundings, the quotient 4: R.  Sums of P add a rounding for each addition
on the way (rows of a warp, 32 warps, the CTAs' results)."""
import numpy as np
import pytest
import torch

from oracle import ends as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": U}     # (bf16 keeps 8 bits, f16 11)


def store(a, dtype, pad=0, lead=0):
    """A device tensor of the values, rounded to `dtype`; pad: wider rows, lead: an unaligned start."""
    T, E = a.shape
    flat = torch.zeros(lead + T * (E + pad), dtype=DT[dtype], device="cuda")
    t = flat[lead:].view(T, E + pad)[:, :E]
    t.copy_(torch.from_numpy(a.astype(np.float32)))
    return t


def f64(t):
    return t.detach().cpu().double().numpy()


def router(T, E, k, seed, dtype="f32", pad=0, lead=0, spread=1.5):
    rng = np.random.default_rng(seed)
    z = store(rng.normal(0, spread, (T, E)), dtype, pad, lead)
    ids = np.argsort(-f64(z), 1, kind="stable")[:, :k].astype(np.int32)
    return z, ids, torch.from_numpy(np.ascontiguousarray(ids)).cuda(), rng


def p_bound(z):
    E = z.shape[1]
    fin = np.where(np.isfinite(z), z, np.nan)
    D = 1.45 * np.nanmax(np.nanmax(fin, 1) - np.nanmin(fin, 1)) if np.isfinite(z).any() else 0.0
    return 2 * (1.4 * D * U + 4 * U) + (E / 32 + 9) * U


def check_loss(lib, z, ids, zt, it, sequences=None, valid=None, status=0):
    st = None if sequences is None else torch.from_numpy(np.asarray(sequences, np.int32)).cuda()
    vt = None if valid is None else torch.from_numpy(np.asarray(valid)).cuda()
    loss, counts, sums, tokens = lib.moe_balance_loss(zt, it, sequences=st, valid=vt)
    assert lib.nvfp4_status_check() == status
    T = z.shape[0]
    want = O.balance_loss(z, ids, sequences, valid)
    assert np.array_equal(counts.cpu().numpy(), want[1]) and np.array_equal(tokens.cpu().numpy(), want[3])
    tol = p_bound(z) + (T / 4864 + 300) * U
    assert np.all(np.abs(f64(sums) - want[2]) <= tol * want[2] + 1e-38)
    assert np.all(np.abs(f64(loss) - want[0]) <= (tol + 64 * U) * want[0] + 1e-38)
    return loss, counts, sums, tokens, st, vt


def check_gradient(lib, z, ids, zt, it, dtype, dw=None, renormalize=True, dloss=None, parts=None, sequences=None,
                   valid=None, out=None, status=0):
    dwt = None if dw is None else torch.from_numpy(dw.astype(np.float32)).cuda()
    dlt = None if dloss is None else torch.from_numpy(dloss.astype(np.float32)).cuda()
    counts, tokens, st, vt = parts or (None, None, None, None)
    got = lib.moe_router_backward(zt, it, dwt, renormalize, dlt, counts, tokens, st, vt, out=out)
    assert lib.nvfp4_status_check() == status
    want, mag = O.router_backward(
        z, ids, None if dw is None else dw.astype(np.float32), renormalize,
        None if dloss is None else dloss.astype(np.float32), None if counts is None else counts.cpu().numpy(),
        None if tokens is None else tokens.cpu().numpy(), sequences, valid)
    # p twice (p and the sum over p), about 40 roundings of the factors and sums, the result's own
    tol = (2 * p_bound(z) + (z.shape[1] / 32 + 40) * U) * mag + HALF_STEP[dtype] * np.abs(want)
    tol += 2.0 ** -25 if dtype == "f16" else 1e-38
    bad = np.abs(f64(got) - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], f64(got)[bad][:5], want[bad][:5])
    return got


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (64, 8, 2), (128, 128, 8), (129, 33, 5), (1000, 60, 4),
                                   (777, 257, 6), (300, 513, 32), (2001, 1024, 16), (9000, 128, 8), (256, 128, 8),
                                   (257, 128, 8), (128, 256, 4), (129, 256, 4), (32, 1024, 2), (33, 1024, 2)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_one_batch(cuda_lib, T, E, k, dtype):
    zt, ids, it, rng = router(T, E, k, T + E, dtype, pad=3 if E % 2 else 0, lead=1)
    z = f64(zt)
    loss, counts, sums, tokens, *_ = check_loss(cuda_lib, z, ids, zt, it)
    for renormalize in (True, False):
        dw, dl = rng.normal(size=(T, k)), rng.normal(size=1)
        parts = (counts, tokens, None, None)
        check_gradient(cuda_lib, z, ids, zt, it, dtype, dw, renormalize, dl, parts)
        check_gradient(cuda_lib, z, ids, zt, it, dtype, dw, renormalize)
    check_gradient(cuda_lib, z, ids, zt, it, dtype, dloss=rng.normal(size=1), parts=(counts, tokens, None, None))


@pytest.mark.parametrize("T,E,k,S", [(50, 16, 2, 7), (400, 128, 8, 64), (5000, 61, 4, 37), (5000, 300, 6, 3)])
def test_sequences_of_any_length(cuda_lib, T, E, k, S):
    """Empty sequences, sequences of one token, tokens before the first and behind the last, padding inside: its
    rows hold NaN, which reaches nothing."""
    zt, ids, it, rng = router(T, E, k, S)
    valid = rng.random(T) < 0.8
    zt[torch.from_numpy(~valid).cuda()] = float("nan")
    z = f64(zt)
    cuts = np.sort(rng.integers(2, T - 1, S + 1)).astype(np.int32)
    cuts[S // 2] = cuts[S // 2 - 1]                                 # an empty one
    if S > 4:
        cuts[1] = cuts[0] + 1                                       # one token
        cuts = np.maximum.accumulate(cuts)
    zz = np.where(valid[:, None], z, 0.0)
    for v in (valid, valid.astype(np.uint8)):
        loss, counts, sums, tokens, st, vt = check_loss(cuda_lib, zz, ids, zt, it, cuts, v)
    assert not torch.isnan(loss).any()
    dl, clean = rng.normal(size=S), torch.from_numpy(np.where(valid[:, None], z, 0.0)).float().cuda()
    got = check_gradient(cuda_lib, zz, ids, clean, it, "f32", rng.normal(size=(T, k)), True, dl,
                         (counts, tokens, st, vt), cuts, valid)
    assert torch.isfinite(got).all()


def test_excluded_experts_and_rows_without_any(cuda_lib):
    T, E, k = 200, 40, 4
    zt, _, _, rng = router(T, E, k, 5)
    drop = torch.from_numpy(rng.random((T, E)) < 0.4).cuda()
    zt.masked_fill_(drop, float("-inf"))
    zt[7] = float("-inf")
    z = f64(zt)
    ids = np.argsort(-z, 1, kind="stable")[:, :k].astype(np.int32)
    it = torch.from_numpy(np.ascontiguousarray(ids)).cuda()
    _, counts, _, tokens, *_ = check_loss(cuda_lib, z, ids, zt, it)
    for renormalize in (True, False):
        got = check_gradient(cuda_lib, z, ids, zt, it, "f32", rng.normal(size=(T, k)), renormalize, rng.normal(size=1),
                             (counts, tokens, None, None))
        assert (got[torch.isneginf(zt)] == 0).all()


def test_infinity_and_nan_stay_in_their_row_and_sequence(cuda_lib):
    T, E, k = 60, 16, 2
    zt, ids, it, rng = router(T, E, k, 6)
    zt[10, 3], zt[31, 0] = float("nan"), float("inf")
    cuts = torch.tensor([0, 20, 30, 40, 60], dtype=torch.int32, device="cuda")
    loss, counts, _, tokens = cuda_lib.moe_balance_loss(zt, it, sequences=cuts)
    assert torch.isnan(loss).tolist() == [True, False, True, False]
    d = cuda_lib.moe_router_backward(zt, it, torch.ones(T, k, device="cuda"), True, torch.ones(4, device="cuda"), counts,
                                     tokens, cuts)
    bad = torch.isnan(d).any(1)
    assert bad[10] and bad[31] and bad.sum() == 2
    assert cuda_lib.nvfp4_status_check() == 0


def test_far_logits(cuda_lib):
    """Chosen experts far below the row's largest: their weights come from their own maximum."""
    z = np.full((3, 64), -300.0)
    z[:, 0] = [0.0, 50.0, 1000.0]
    z[:, 5], z[:, 9] = -120.0, -121.0
    ids = np.array([[5, 9]] * 3, np.int32)
    zt, it = store(z, "f32"), torch.from_numpy(ids).cuda()
    dw = np.array([[1.0, -2.0]] * 3)
    got = f64(cuda_lib.moe_router_backward(zt, it, torch.from_numpy(dw).float().cuda()))
    want, _ = O.router_backward(z, ids, dw)
    assert np.abs(got - want).max() <= 2.0 ** -18


def test_ids_twice_and_outside(cuda_lib):
    T, E, k = 40, 70, 6
    zt, ids, it, rng = router(T, E, k, 8)
    ids[3] = [9, 9, 9, 1, 2, 9]
    ids[17, 2] = ids[17, 5]
    ids[20, 1], ids[21, 0], ids[39, 5] = -1, E, 2 ** 31 - 1
    it.copy_(torch.from_numpy(ids))
    z = f64(zt)
    _, counts, _, tokens, *_ = check_loss(cuda_lib, z, ids, zt, it, status=cuda_lib.Status.DEVICE_STATUS)
    for renormalize in (True, False):
        check_gradient(cuda_lib, z, ids, zt, it, "f32", rng.normal(size=(T, k)), renormalize, rng.normal(size=1),
                       (counts, tokens, None, None), status=cuda_lib.Status.DEVICE_STATUS)


@pytest.mark.parametrize("cuts", [[0, 9, 5, 20], [-1, 9, 20, 20], [0, 9, 20, 21], [30, 31, 40, 50]])
def test_sequences_that_descend_or_leave_the_batch(cuda_lib, cuts):
    zt, ids, it, _ = router(20, 8, 2, 9)
    st = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    loss, counts, _, tokens = cuda_lib.moe_balance_loss(zt, it, sequences=st)
    assert cuda_lib.nvfp4_status_check() == cuda_lib.Status.DEVICE_STATUS
    bad = [a < 0 or b < a or b > 20 for a, b in zip(cuts[:-1], cuts[1:])]
    assert torch.isnan(loss).tolist() == bad
    one = torch.tensor([cuts[1], cuts[0]], dtype=torch.int32, device="cuda")   # a single sequence, as well
    assert torch.isnan(cuda_lib.moe_balance_loss(zt, it, sequences=one)[0]).all()
    assert cuda_lib.nvfp4_status_check() == cuda_lib.Status.DEVICE_STATUS
    cuda_lib.moe_router_backward(zt, it, dloss=torch.ones(3, device="cuda"), counts=counts, tokens=tokens, sequences=st)
    cuda_lib.nvfp4_status_check()


def test_in_place_views_and_empty_batches(cuda_lib):
    T, E, k = 90, 24, 3
    zt, ids, it, rng = router(T, E, k, 10, "bf16", pad=5, lead=1)
    dw = torch.from_numpy(rng.normal(size=(T, 2 * k))).float().cuda()[:, ::2]        # strided companions
    want = cuda_lib.moe_router_backward(zt.contiguous(), it, dw.contiguous())
    assert torch.equal(cuda_lib.moe_router_backward(zt, it, dw, out=zt), want) and torch.equal(zt, want)
    e = torch.empty(0, E, device="cuda")
    i = torch.empty(0, k, dtype=torch.int32, device="cuda")
    for S, st in ((1, None), (3, torch.zeros(4, dtype=torch.int32, device="cuda"))):
        out = cuda_lib.moe_balance_loss(e, i, sequences=st)
        assert [tuple(o.shape) for o in out] == [(S,), (S, E), (S, E), (S,)] and all((o == 0).all() for o in out)
    assert cuda_lib.moe_router_backward(e, i, torch.empty(0, k, device="cuda")).shape == (0, E)
    # every token is padding, or belongs to nobody
    none = torch.zeros(T, dtype=torch.bool, device="cuda")
    assert (cuda_lib.moe_balance_loss(want, it, valid=none)[0] == 0).all()
    out = cuda_lib.moe_balance_loss(want, it, sequences=torch.tensor([T, T], dtype=torch.int32, device="cuda"))
    assert all((o == 0).all() for o in out)
    d = cuda_lib.moe_router_backward(want, it, dloss=torch.ones(1, device="cuda"), counts=out[1], tokens=out[3], valid=none)
    assert (d == 0).all() and cuda_lib.nvfp4_status_check() == 0


def test_counts_of_several_devices(cuda_lib):
    """Two halves of a batch with the counts and tokens of both: the gradient of the whole batch's loss."""
    T, E, k = 256, 32, 4
    zt, ids, it, _ = router(T, E, k, 11)
    _, counts, sums, tokens = cuda_lib.moe_balance_loss(zt, it)
    halves = [cuda_lib.moe_balance_loss(zt[h], it[h]) for h in (slice(0, 128), slice(128, T))]
    assert torch.equal(halves[0][1] + halves[1][1], counts) and torch.equal(halves[0][3] + halves[1][3], tokens)
    assert torch.allclose(halves[0][2] + halves[1][2], sums, rtol=2 ** -18)
    one = torch.full((1,), 0.7, device="cuda")
    whole = cuda_lib.moe_router_backward(zt, it, dloss=one, counts=counts, tokens=tokens)
    for h in (slice(0, 128), slice(128, T)):
        assert torch.equal(cuda_lib.moe_router_backward(zt[h], it[h], dloss=one, counts=counts, tokens=tokens), whole[h])


def test_streams_and_graphs(cuda_lib):
    """A given stream, and a captured forward and backward that replay on new inputs; two graphs of one workspace,
    one after the other, give what eager calls give."""
    T, E, k = 3000, 128, 8
    zt, ids, it, rng = router(T, E, k, 12)
    dw = torch.from_numpy(rng.normal(size=(T, k))).float().cuda()
    one = torch.ones(1, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def step():
        loss, counts, sums, tokens = cuda_lib.moe_balance_loss(zt, it, workspace=ws)
        return loss, counts, sums, tokens, cuda_lib.moe_router_backward(zt, it, dw, True, one, counts, tokens)

    want = [o.clone() for o in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cuda_lib.moe_balance_loss(zt, it, stream=side)
    d = cuda_lib.moe_router_backward(zt, it, dw, True, one, got[1], got[3], stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, d), want))
    graphs = []
    for _ in range(2):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    other = store(np.random.default_rng(13).normal(size=(T, E)), "f32")
    for z in (zt.clone(), other):
        zt.copy_(z)
        want = [o.clone() for o in step()]
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert cuda_lib.nvfp4_status_check() == 0


def test_the_router_s_own_path(cuda_lib):
    """Weights and ids of moe_route_topk, the gradient by moe_expert_backward's dw: against differences in float64
    of the weights as a function of the logits."""
    T, E, k = 64, 16, 4
    zt, _, _, rng = router(T, E, k, 14)
    ids, w = cuda_lib.moe_route_topk(zt.contiguous(), k)
    want_w = O.route_weights(f64(zt), ids.cpu().numpy())
    assert np.abs(f64(w) - want_w).max() < 2.0 ** -20
    dw = torch.from_numpy(rng.normal(size=(T, k))).float().cuda()
    got = f64(cuda_lib.moe_router_backward(zt, ids, dw))
    z, n, dwn = f64(zt), ids.cpu().numpy(), f64(dw)
    step = rng.normal(size=z.shape)
    f = lambda h: (O.route_weights(z + h * step, n) * dwn).sum()  # noqa: E731
    assert abs((f(1e-5) - f(-1e-5)) / 2e-5 - (got * step).sum()) < 2.0 ** -16 * np.abs(got * step).sum()
