"""GPU parity of the operators on rows of logits (token_logprobs, distill_topk and their
backwards) with the float64 oracle.

Bounds.  u = 2^-24.  A thread adds its chunks of a slice one after the other and the rest
of the sum is a tree, so a sum of exponentials is off by at most D u of itself, with
D = chunks a thread + 24 (the chunk's 8, 5 + 1 + 5 steps of the trees, the rescalings); an
exponential itself by 4 u (the hardware's 2^-22) plus the rounding of its argument, 2 |t| u
for an argument of t, where terms with |t| > 40 no longer matter: 80 u.  So ln sum is off by
eps = (D + 84) u, and lse by 2 u |lse| more.  The entropy ln s - E[t] adds the same
relative errors of the terms times E|t| <= ln V.  A probability recomputed from lse is off by
eps + 2 u |lse| + 84 u + its argument's rounding, relatively.  Outputs in 16 bits add half a
unit in the last place."""
import numpy as np
import pytest
import torch

from oracle import learner as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}


def eps(V):
    slices = 8 if V >= 65536 else 4 if V >= 32768 else 2 if V >= 16384 else 1
    return (V / 8 / 256 / slices + 1 + 24 + 84) * U


def store(z, dtype, pad=0, lead=0):
    """z as a view [:, :V] of storage with `pad` more columns, starting `lead` elements in."""
    T, V = z.shape
    flat = torch.full((lead + T * (V + pad),), float("nan"), dtype=DT[dtype], device="cuda")
    view = flat[lead:].view(T, V + pad)[:, :V]
    view.copy_(torch.from_numpy(z))
    return view


def f64(t):
    return t.detach().double().cpu().numpy()


def logits(T, V, seed, masked=0.0, std=2.5):
    rng = np.random.default_rng(seed)
    z = rng.normal(0.0, std, (T, V))
    z[np.arange(T), rng.integers(0, V, T)] += 8.0
    if masked:
        z[rng.random((T, V)) < masked] = -np.inf
        z[np.arange(T), rng.integers(0, V, T)] = 1.0
    return z, rng


def near(got, ref, bound):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        bad = ~same & ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4], np.broadcast_to(bound, ref.shape)[bad][:4])


def check_forward(lib, zt, y, scale, k):
    got = lib.token_logprobs(zt, None if y is None else torch.from_numpy(y).cuda(), top_k=k, scale=scale)
    assert lib.nvfp4_status_check() == 0
    z = f64(zt)
    V = z.shape[1]
    s = float(np.float32(scale))
    ref = O.token_logprobs(z, y, s, k)
    e = eps(V)
    lse_bound = e + 2 * U * np.abs(ref["lse"])
    near(got[1].cpu(), ref["lse"], lse_bound)
    near(got[2].cpu(), ref["entropy"], e * (1 + 2 * np.log(V)) + 2 * U * (ref["entropy"] + np.log(V)))
    if y is not None:
        near(got[0].cpu(), ref["logprob"], e + 4 * U * np.abs(ref["logprob"]) + 2 * U * np.log(V))
    if k:
        np.testing.assert_array_equal(got[4].cpu().numpy(), ref["top_ids"])
        near(got[3].cpu(), ref["top_logprob"], e + 4 * U * np.abs(ref["top_logprob"]) + 2 * U * np.log(V))
    return got, ref


# one token; less than a chunk; one chunk; odd; around the numbers of slices; several rows
# each with the rows of one cluster or, from 608 rows on, one CTA a row
SHAPES = [(1, 1, 1), (3, 7, 7), (2, 8, 3), (5, 1000, 20), (4, 1003, 128), (2, 4097, 5), (3, 8191, 20), (3, 8192, 20),
          (2, 16389, 64), (2, 32767, 128), (3, 32768, 20), (2, 50021, 128), (1, 131072, 20), (700, 1003, 5),
          (640, 33001, 20)]


@pytest.mark.parametrize("T,V,k", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_forward(cuda_lib, T, V, k, dtype):
    z, rng = logits(T, V, T + V)
    y = rng.integers(0, V, T).astype(np.int32)
    y[T // 2] = -100 if T > 2 else y[T // 2]
    check_forward(cuda_lib, store(z, dtype), y, 1.0, k)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,lead", [(0, 1), (5, 3), (8, 0), (1, 7)])
def test_forward_strides_masks_and_scale(cuda_lib, dtype, pad, lead):
    z, rng = logits(9, 10007, pad + 10 * lead, masked=0.4)
    z[3, :] = -np.inf                                  # a row whose mask leaves nothing
    z[4, :] = -np.inf
    z[4, 17:20] = [0.5, 2.0, 0.5]                      # fewer allowed tokens than alternatives
    y = rng.integers(0, 10007, 9).astype(np.int32)
    y[4], y[5] = 17, -100
    got, ref = check_forward(cuda_lib, store(z, dtype, pad, lead), y, 1.7, 20)
    assert np.isneginf(got[1][3].item()) and np.isneginf(got[0][3].item()) and got[2][3].item() == 0
    assert got[4][4].tolist()[:4] == [18, 17, 19, -1]


def test_no_targets_no_entropy(cuda_lib):
    z, _ = logits(4, 3001, 5)
    zt = store(z, "bf16")
    lp, lse, ent, top, ids = cuda_lib.token_logprobs(zt, entropy=False)
    assert lp is None and ent is None and top is None and ids is None
    near(lse.cpu(), O.token_logprobs(f64(zt))["lse"], eps(3001) + 2 * U * 20)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_lowest_values_and_ties(cuda_lib, dtype):
    """Rows of the type's lowest value are uniform; equal values (and the two zeros) rank by id."""
    low = float(torch.finfo(DT[dtype]).min)
    V = 9001
    z = np.full((5, V), low)
    z[1, ::3] = 0.0
    z[1, 1::6] = -0.0
    z[2, :] = 0.25
    z[3, 5000:5040] = 4.0
    z[4, ::-1] = np.repeat(np.arange(V // 100 + 1), 100)[:V]       # plateaus, best last
    y = np.array([7, 1, 8999, 5039, 0], np.int32)
    check_forward(cuda_lib, store(z, dtype), y, 1.0, 128)


def test_rows_of_lowest_values_backward(cuda_lib):
    """A mask of the type's lowest value that leaves nothing: distillation sees a uniform row; the
    log probabilities' gradient, recomputed from lse, is zero."""
    low = float(torch.finfo(torch.bfloat16).min)
    z, rng = logits(3, 4001, 12)
    z[1, :] = low
    z[2, 50:] = low
    zt = store(z, "bf16")
    ids, val = teacher(3, 4001, 12, rng)
    ids[2] = np.arange(12)
    for tail in (False, True):
        check_distill(cuda_lib, zt, ids, val, tail)
    y = torch.zeros(3, dtype=torch.int32, device="cuda")
    _, lse, _, _, _ = cuda_lib.token_logprobs(zt, y)
    d = cuda_lib.token_logprobs_backward(zt, lse, y, torch.ones(3, device="cuda"))
    assert d[0].any() and not d[1].any() and d[2].any() and not d[2, 50:].any()


def test_candidates_beyond_one_round(cuda_lib):
    """A few threads' cells hold everything large (chunks 256 apart): many more candidates than the
    list, so the bounded buffer has to keep the best between rounds."""
    V, T = 1 << 20, 2
    rng = np.random.default_rng(9)
    z = rng.normal(0.0, 1.0, (T, V))
    chunk = np.arange(V // 8)
    hot = (chunk % 256) < 100
    zz = z.reshape(T, V // 8, 8)
    zz[:, hot, :] += 40.0
    check_forward(cuda_lib, store(z, "f32"), np.array([0, V - 1], np.int32), 1.0, 128)
    check_forward(cuda_lib, store(z, "bf16"), np.array([0, V - 1], np.int32), 1.0, 128)
    # the same with one CTA a row
    V, T = 40000, 640
    z = rng.normal(0.0, 1.0, (T, V))
    z.reshape(T, V // 8, 8)[:, (np.arange(V // 8) % 256) < 100, :] += 40.0
    check_forward(cuda_lib, store(z, "f32"), np.zeros(T, np.int32), 1.0, 128)


@pytest.mark.parametrize("T", [2, 640])
def test_few_threads_hold_everything(cuda_lib, T):
    """All but 100 threads' chunks excluded: fewer threads than alternatives, many candidates each."""
    V = 40000
    rng = np.random.default_rng(T)
    z = np.full((T, V), -np.inf)
    hot = (np.arange(V // 8) % 256) < 100
    z.reshape(T, V // 8, 8)[:, hot, :] = rng.normal(0.0, 1.0, (T, hot.sum(), 8))
    check_forward(cuda_lib, store(z, "f16"), np.zeros(T, np.int32), 1.0, 128)


def test_no_rows(cuda_lib):
    z = torch.empty(0, 64, device="cuda")
    i, f = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    got = cuda_lib.token_logprobs(z, i, top_k=3)
    assert [t.shape for t in got] == [(0,), (0,), (0,), (0, 3), (0, 3)]
    assert cuda_lib.token_logprobs_backward(z, f, i, f).shape == (0, 64)
    ids, val = torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda")
    assert cuda_lib.distill_topk(z, ids, val)[0].shape == (0,)
    assert cuda_lib.distill_topk_backward(z, ids, val)[1].shape == (0, 64)


def test_not_a_number_rows(cuda_lib):
    z, _ = logits(3, 5000, 11)
    z[0, 4999] = np.nan
    z[1, 0] = np.inf
    lp, lse, ent, top, ids = cuda_lib.token_logprobs(store(z, "f32"), torch.zeros(3, dtype=torch.int32, device="cuda"),
                                                     top_k=4)
    assert torch.isnan(lse[:2]).all() and torch.isnan(lp[:2]).all() and torch.isnan(ent[:2]).all()
    assert torch.isfinite(lse[2]) and torch.isfinite(top[2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_rows_bits_do_not_depend_on_the_batch(cuda_lib, dtype):
    """The same row alone, among 700 others, and at every alignment: the same bits."""
    V = 33003
    z, rng = logits(700, V, 21)
    y = torch.from_numpy(rng.integers(0, V, 700).astype(np.int32)).cuda()
    ids = torch.from_numpy(np.stack([rng.permutation(V)[:30] for _ in range(700)]).astype(np.int32)).cuda()
    val = torch.log_softmax(torch.randn(700, 31, generator=torch.Generator().manual_seed(1)), 1)[:, :30].cuda()
    zt = store(z, dtype)
    many = cuda_lib.token_logprobs(zt, y, top_k=20)
    loss = [cuda_lib.distill_topk(zt, ids, val, tail) for tail in (False, True)]
    for r in (0, 1, 350, 699):
        for lead in (0, 1, 2, 3):
            one = store(z[r:r + 1], dtype, lead=lead)
            alone = cuda_lib.token_logprobs(one, y[r:r + 1], top_k=20)
            for a, b in zip(many, alone):
                assert torch.equal(a[r:r + 1], b)
            for tail in (False, True):
                for a, b in zip(loss[tail], cuda_lib.distill_topk(one, ids[r:r + 1], val[r:r + 1], tail)):
                    assert torch.equal(a[r:r + 1], b)


# ------------------------------------------------------------------------------- backward

def check_backward(lib, zt, y, g, h, scale, out=None):
    T, V = zt.shape
    yt = None if y is None else torch.from_numpy(y).cuda()
    z = f64(zt)
    _, lse, ent, _, _ = lib.token_logprobs(zt, yt, scale=scale)
    gt = None if g is None else torch.from_numpy(g.astype(np.float32)).cuda()
    ht = None if h is None else torch.from_numpy(h.astype(np.float32)).cuda()
    got = lib.token_logprobs_backward(zt, lse, yt, gt, entropy=ent if h is not None else None, dentropy=ht,
                                      scale=scale, out=out)
    assert lib.nvfp4_status_check() == 0
    s = float(np.float32(scale))
    g64 = None if g is None else g.astype(np.float32).astype(np.float64)
    h64 = None if h is None else h.astype(np.float32).astype(np.float64)
    ref = O.token_logprobs_backward(z, y, g64, h64, s)
    lp, p, l = O.softmax_stats(z * s)
    alp = np.where(p > 0, np.abs(np.where(p > 0, lp, 0.0)), 0.0)
    G = 0.0 if g is None else np.abs(g64)[:, None]
    H = 0.0 if h is None else np.abs(h64)[:, None]
    al = np.where(np.isfinite(l), np.abs(l), 0.0)[:, None]
    rel = eps(V) + 2 * U * al + 84 * U + 4 * U * (alp + al)
    size = p * (G + H * (alp + np.log(V) + 1))
    bound = s * (size * rel + H * p * eps(V) * (2 + 2 * np.log(V))) + HALF_ULP[zt.dtype] * 1.01 * np.abs(ref)
    bound = bound + 4 * U * s * G * (ref > 0) + TINY[zt.dtype] + s * 1e-37
    near(f64(got), ref, bound)
    return got


@pytest.mark.parametrize("T,V", [(1, 1), (3, 7), (2, 1000), (4, 1003), (2, 16384), (3, 16385), (2, 50021), (40, 4096)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("entropy", [False, True])
def test_backward(cuda_lib, T, V, dtype, entropy):
    z, rng = logits(T, V, 3 * T + V)
    y = rng.integers(0, V, T).astype(np.int32)
    if T > 2:
        y[1] = -100
    check_backward(cuda_lib, store(z, dtype), y, rng.normal(size=T), rng.normal(size=T) if entropy else None, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,lead,opad,olead", [(0, 1, 0, 1), (3, 0, 3, 0), (0, 0, 1, 3), (5, 2, 8, 0)])
def test_backward_strides_masks_in_place(cuda_lib, dtype, pad, lead, opad, olead):
    z, rng = logits(7, 6007, 17, masked=0.5)
    z[2, :] = -np.inf
    z[3, 100] = -np.inf
    y = rng.integers(0, 6007, 7).astype(np.int32)
    y[3], y[4] = 100, -100                             # an excluded target; an ignored row
    g, h = rng.normal(size=7), rng.normal(size=7)
    zt = store(z, dtype, pad, lead)
    out = store(np.zeros_like(z), dtype, opad, olead)
    got = check_backward(cuda_lib, zt, y, g, h, 0.6, out=out)
    assert not got[2].any() and not got[4].any() and got[3, 100] == 0
    keep = got.clone()
    same = check_backward(cuda_lib, zt.clone(), y, g, h, 0.6)
    assert torch.equal(same, keep)
    # in place, in storage whose padding must survive
    flat = torch.zeros(lead + 7 * (6007 + pad), dtype=zt.dtype, device="cuda")
    view = flat[lead:].view(7, 6007 + pad)[:, :6007]
    view.copy_(torch.from_numpy(z))
    _, lse, ent, _, _ = cuda_lib.token_logprobs(view, torch.from_numpy(y).cuda(), scale=0.6)
    f = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()
    cuda_lib.token_logprobs_backward(view, lse, torch.from_numpy(y).cuda(), f(g), entropy=ent, dentropy=f(h), scale=0.6,
                                     out=view)
    assert torch.equal(view, keep)
    assert not flat[:lead].any() and not flat[lead:].view(7, 6007 + pad)[:, 6007:].any()


def test_entropy_alone_and_bad_target(cuda_lib):
    z, rng = logits(3, 999, 2)
    check_backward(cuda_lib, store(z, "f32"), None, None, rng.normal(size=3), 1.0)
    zt = store(z, "f32")
    y = torch.tensor([5, 999, -3], dtype=torch.int32, device="cuda")
    lp, lse, _, _, _ = cuda_lib.token_logprobs(zt, y)
    assert cuda_lib.nvfp4_status_check() == cuda_lib.Status.DEVICE_STATUS
    assert torch.isfinite(lp[0]) and torch.isnan(lp[1:]).all() and torch.isfinite(lse).all()
    d = cuda_lib.token_logprobs_backward(zt, lse, y, torch.ones(3, device="cuda"))
    assert d[0].any() and not d[1:].any()


def test_gradient_by_differences(cuda_lib):
    """Central differences of the forward's own outputs along random directions."""
    z, rng = logits(6, 2003, 8)
    y = torch.from_numpy(rng.integers(0, 2003, 6).astype(np.int32)).cuda()
    zt = store(z, "f32")
    g, h = (torch.randn(6, generator=torch.Generator().manual_seed(s)).cuda() for s in (1, 2))
    _, lse, ent, _, _ = cuda_lib.token_logprobs(zt, y)
    d = cuda_lib.token_logprobs_backward(zt, lse, y, g, entropy=ent, dentropy=h)
    ids = torch.from_numpy(np.stack([rng.permutation(2003)[:40] for _ in range(6)]).astype(np.int32)).cuda()
    val = torch.log_softmax(torch.randn(6, 60, generator=torch.Generator().manual_seed(5)), 1)[:, :40].cuda()
    w = g.abs()
    step = 2.0 ** -5

    def value(x):
        lp, _, en, _, _ = cuda_lib.token_logprobs(x, y)
        return (g * lp + h * en).double().sum().item()

    for seed in range(3):
        dirn = torch.randn(zt.shape, generator=torch.Generator().manual_seed(10 + seed)).cuda()
        num = (value(zt + step * dirn) - value(zt - step * dirn)) / (2 * step)
        want = (d.double() * dirn.double()).sum().item()
        # float32 values of size ~30 give 1e-5 / step; the third derivative step^2 / 6 of size ~10
        assert abs(num - want) < 6 * 4e-6 / step + step ** 2 * 10
        for tail in (False, True):
            _, dd = cuda_lib.distill_topk_backward(zt, ids, val, w, tail)
            lo = lambda x: (w * cuda_lib.distill_topk(x, ids, val, tail)[0]).double().sum().item()
            num = (lo(zt + step * dirn) - lo(zt - step * dirn)) / (2 * step)
            assert abs(num - (dd.double() * dirn.double()).sum().item()) < 6 * 4e-6 / step + step ** 2 * 10


# ------------------------------------------------------------------------------- distillation

def teacher(T, V, K, rng, short=False, mass=0.8):
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)]).astype(np.int32)
    t = rng.normal(0.0, 2.0, (T, K))
    t = t - np.log(np.exp(t).sum(1, keepdims=True)) + np.log(mass)
    if short:
        for r in range(T):
            ids[r, rng.integers(0, K + 1):] = -1
    return ids, t.astype(np.float32)


def check_distill(lib, zt, ids, val, tail, scale=1.0, w=None, out=None):
    T, V = zt.shape
    it, vt = torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda()
    z = f64(zt)
    s = float(np.float32(scale))
    ref, grad, ref_lse = O.distill(z, ids, val, tail, s)
    lp, p, l = O.softmax_stats(z * s)
    e = eps(V)
    with np.errstate(invalid="ignore", over="ignore"):
        al = np.where(np.isfinite(l), np.abs(l), 0.0)
    q = np.where(ids >= 0, np.exp(val.astype(np.float64)), 0.0)
    if not tail:
        q = q / np.maximum(q.sum(1, keepdims=True), 1e-300)
    at = np.take_along_axis(lp, np.clip(ids, 0, V - 1), 1)
    use = (q > 0) & np.isfinite(at)
    terms = np.where(use, q * (np.abs(np.log(np.where(use, q, 1.0))) + np.abs(np.where(use, at, 0.0)) + 1), 0.0).sum(1)
    K = ids.shape[1]
    bound = 2 * e + (16 + K / 8) * U * (terms + 2 * al + 20)
    rest = np.ones_like(p, bool)
    for t in range(T):
        rest[t, ids[t][ids[t] >= 0]] = False
    pr = np.where(rest, p, 0.0).sum(1)
    qr = np.maximum(0.0, 1.0 - q.sum(1))
    if tail:   # q_r carries the rounding of the listed sum: (K/8 + 16) u
        lpr = np.abs(np.log(np.where(pr > 0, pr, 1.0)))
        lqr = np.abs(np.log(np.maximum(qr, U)))
        bound = bound + (K / 8 + 16) * U * (lpr + lqr + 2) + qr * (e + 4 * U * al)
    loss, lse = lib.distill_topk(zt, it, vt, tail, scale)
    near(loss.cpu(), ref, bound)
    near(lse.cpu(), ref_lse, 2 * e + 2 * U * al)
    wt = None if w is None else torch.from_numpy(w.astype(np.float32)).cuda()
    loss2, d = lib.distill_topk_backward(zt, it, vt, wt, tail, scale, out=out)
    assert lib.nvfp4_status_check() == 0
    assert torch.equal(loss2.nan_to_num(nan=-1.0), loss.nan_to_num(nan=-1.0))
    w64 = np.ones(T) if w is None else w.astype(np.float32).astype(np.float64)
    want = grad * w64[:, None]
    alp = np.where(p > 0, np.abs(np.where(p > 0, lp, 0.0)), 0.0)
    rel = 2 * e + 2 * U * al[:, None] + 84 * U + 4 * U * (alp + al[:, None])
    qfull = np.zeros_like(p)
    for t in range(T):
        live = ids[t] >= 0
        qfull[t, ids[t][live]] = q[t][live]
    size = p * rel + qfull * (K / 8 + 16) * U
    if tail:
        cond = np.where(rest & (pr > 0)[:, None], p / np.where(pr > 0, pr, 1.0)[:, None], 0.0)
        lr = np.abs(np.log(np.where(pr > 0, pr, 1.0)))[:, None]
        size = size + cond * ((pr + qr)[:, None] * (rel + 4 * U * lr) + (K / 8 + 16) * U)
    gb = s * np.abs(w64)[:, None] * size + HALF_ULP[zt.dtype] * 1.01 * np.abs(want) + TINY[zt.dtype] + 1e-37
    near(f64(d), want, gb)
    return loss, d


@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (3, 7, 5), (2, 1000, 128), (5, 1003, 17), (3, 8192, 64), (2, 16389, 1),
                                   (3, 32768, 100), (2, 50021, 128), (620, 1003, 9)])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_distill(cuda_lib, T, V, K, tail, dtype):
    z, rng = logits(T, V, T + V + K)
    ids, val = teacher(T, V, K, rng, short=T > 4)
    check_distill(cuda_lib, store(z, dtype), ids, val, tail, w=rng.normal(size=T))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,V", [("f32", 300007), ("bf16", 1 << 20), ("f32", (1 << 20) - 3)])
def test_distill_long_rows(cuda_lib, tail, dtype, V):
    """Slices that fill the shared memory, and slices that do not fit into it; in place too."""
    z, rng = logits(2, V, V)
    ids, val = teacher(2, V, 100, rng)
    zt = store(z, dtype, lead=1)
    _, d = check_distill(cuda_lib, zt, ids, val, tail)
    keep = d.clone()
    cuda_lib.distill_topk_backward(zt, torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda(), tail=tail, out=zt)
    assert torch.equal(zt, keep)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,T,V", [("bf16", 2500, 8200), ("f16", 1900, 20003), ("f32", 700, 33001), ("f32", 2000, 16400)])
def test_distill_many_rows(cuda_lib, tail, dtype, T, V):
    """Several rows a cluster, several slices a CTA: every row equals the same row alone."""
    z, rng = logits(64, V, V + T)
    ids, val = teacher(64, V, 37, rng, short=True)
    pick = torch.from_numpy(rng.integers(0, 64, T)).cuda()
    zt, it, vt = store(z, dtype), torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda()
    w = torch.ones(T, device="cuda")
    few_loss, few = cuda_lib.distill_topk_backward(zt, it, vt, w[:64], tail)
    check_distill(cuda_lib, zt, ids, val, tail)
    many = torch.full((T, V + 5), -1.0, dtype=DT[dtype], device="cuda")
    many[:, :V] = zt[pick]
    for x in (many[:, :V], many[:, :V].contiguous()):
        loss, d = cuda_lib.distill_topk_backward(x, it[pick], vt[pick], w, tail)
        assert torch.equal(loss, few_loss[pick]) and torch.equal(d, few[pick])
    cuda_lib.distill_topk_backward(many[:, :V], it[pick], vt[pick], w, tail, out=many[:, :V])
    assert torch.equal(many[:, :V], few[pick]) and (many[:, V:] == -1).all()
    assert cuda_lib.nvfp4_status_check() == 0


def test_distill_student_without_tokens(cuda_lib):
    z = np.full((2, 5000), -np.inf)
    z[1, 7] = 1.0
    ids = np.array([[7, 9], [7, -1]], np.int32)
    val = np.log(np.array([[0.5, 0.25], [1.0, 1.0]])).astype(np.float32)
    for tail in (False, True):
        loss, d = cuda_lib.distill_topk_backward(store(z, "f32"), torch.from_numpy(ids).cuda(),
                                                 torch.from_numpy(val).cuda(), tail=tail)
        assert loss.tolist() == [float("inf"), 0.0] and not d.any()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,lead", [(0, 0), (3, 5)])
def test_distill_masks_and_in_place(cuda_lib, tail, dtype, pad, lead):
    T, V, K = 8, 9003, 20
    z, rng = logits(T, V, 31, masked=0.5)
    ids, val = teacher(T, V, K, rng)
    z[np.arange(T)[:, None], ids] = rng.normal(0, 2, (T, K))       # the mask spares the teacher's tokens
    z[1, ids[1, 3]] = -np.inf                                     # but one: infinite loss
    val[2, 5] = -np.inf                                           # an entry without mass
    ids[3, :] = -1                                                # no entries
    z[4, :] = -np.inf                                             # nothing outside the list
    z[4, ids[4]] = rng.normal(0, 2, K)
    z[5, :] = -40.0                                               # next to nothing outside the list
    z[5, ids[5]] = 30.0
    zt = store(z, dtype, pad, lead)
    loss, d = check_distill(cuda_lib, zt, ids, val, tail, 1.3, rng.normal(size=T))
    assert torch.isinf(loss[1]) and loss[3] == 0 and not d[3].any()
    w = torch.ones(T, device="cuda")
    it, vt = torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda()
    keep = cuda_lib.distill_topk_backward(zt, it, vt, w, tail, 1.3)[1]
    flat = torch.zeros(lead + T * (V + pad), dtype=zt.dtype, device="cuda")
    view = flat[lead:].view(T, V + pad)[:, :V]
    view.copy_(torch.from_numpy(z))
    cuda_lib.distill_topk_backward(view, it, vt, w, tail, 1.3, out=view)
    assert torch.equal(view, keep)
    assert not flat[:lead].any() and not flat[lead:].view(T, V + pad)[:, V:].any()


def test_distill_bad_lists(cuda_lib):
    z, rng = logits(3, 500, 3)
    zt = store(z, "bf16")
    val = torch.zeros(3, 4, device="cuda")
    ids = torch.tensor([[1, 2, 3, -1], [4, 500, 5, 6], [7, 8, 7, 9]], dtype=torch.int32, device="cuda")
    loss, d = cuda_lib.distill_topk_backward(zt, ids, val, tail=False)
    assert cuda_lib.nvfp4_status_check() == cuda_lib.Status.DEVICE_STATUS
    assert torch.isfinite(loss[0]) and d[0].any()
    assert torch.isnan(loss[1:]).all() and not d[1:].any()


def test_teachers_list_feeds_the_student(cuda_lib):
    """token_logprobs' alternatives are distill_topk's teacher; a student equal to the teacher has
    no loss and no gradient, beyond round-off."""
    z, _ = logits(5, 12001, 44)
    zt = store(z, "f32")
    _, _, _, lp, ids = cuda_lib.token_logprobs(zt, top_k=64)
    loss, d = cuda_lib.distill_topk_backward(zt, ids, lp, tail=True)
    assert loss.abs().max().item() < 4 * eps(12001) + 64 * U * 30
    assert d.abs().max().item() < 4 * eps(12001) + 64 * U * 30


def test_largest_offsets(cuda_lib):
    """Rows whose first element lies beyond 2^31: the last rows of a large batch."""
    T, V = 17000, 131072
    zt = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
    zt.fill_(0)
    z, rng = logits(3, V, 77)
    zt[-3:] = torch.from_numpy(z).to(torch.bfloat16).cuda()
    y = torch.full((T,), -100, dtype=torch.int32, device="cuda")
    y[-3:] = torch.tensor([1, 2, 3], dtype=torch.int32)
    got = cuda_lib.token_logprobs(zt, y, top_k=7)
    alone = cuda_lib.token_logprobs(zt[-3:].clone(), y[-3:], top_k=7)
    for a, b in zip(got, alone):
        assert torch.equal(a[-3:], b)
    d = cuda_lib.token_logprobs_backward(zt, got[1], y, torch.ones(T, device="cuda"))
    d1 = cuda_lib.token_logprobs_backward(zt[-3:].clone(), alone[1], y[-3:], torch.ones(3, device="cuda"))
    assert torch.equal(d[-3:], d1) and not d[:5].any()
    del d
    ids = torch.full((T, 3), -1, dtype=torch.int32, device="cuda")
    ids[-3:] = got[4][-3:, :3]
    val = torch.zeros(T, 3, device="cuda")
    loss, dd = cuda_lib.distill_topk_backward(zt, ids, val, tail=False)
    loss1, dd1 = cuda_lib.distill_topk_backward(zt[-3:].clone(), ids[-3:], val[-3:], tail=False)
    assert torch.equal(loss[-3:], loss1) and torch.equal(dd[-3:], dd1) and not dd[:5].any()


def test_another_stream_and_a_graph(cuda_lib):
    z, rng = logits(6, 7001, 5)
    zt = store(z, "bf16")
    y = torch.from_numpy(rng.integers(0, 7001, 6).astype(np.int32)).cuda()
    want = cuda_lib.token_logprobs(zt, y, top_k=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = cuda_lib.token_logprobs(zt, y, top_k=9, stream=s)
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = cuda_lib.token_logprobs(zt, y, top_k=9)
        _, d = cuda_lib.distill_topk_backward(zt, got[4], got[3])
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_copies_belong_to_the_given_stream(cuda_lib):
    """Dense copies of strided companions are read on the given stream, after the call has returned:
    nothing that the current stream allocates meanwhile may take their place."""
    T, V, K = 64, 4001, 8
    z, rng = logits(T, V, 5)
    zt = store(z, "bf16")
    y = torch.from_numpy(rng.integers(1, V, T).astype(np.int32)).cuda()
    _, _, _, values, ids = cuda_lib.token_logprobs(zt, top_k=K)
    strided = lambda t: torch.stack((t, t), -1)[..., 0]
    y2, ids2, values2 = strided(y), strided(ids), strided(values)
    assert not (y2.is_contiguous() or ids2.is_contiguous() or values2.is_contiguous())
    want = cuda_lib.token_logprobs(zt, y2)[0], *cuda_lib.distill_topk_backward(zt, ids2, values2)
    torch.zeros(T, dtype=torch.int32, device="cuda")   # every kernel has run once: loading one could wait
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)   # some 50 ms, in which the other stream gets its work done
    lp = cuda_lib.token_logprobs(zt, y2, stream=s)[0]
    got = lp, *cuda_lib.distill_topk_backward(zt, ids2, values2, None, True, 1.0, None, s)
    others = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (T, T * K) for _ in range(64)]
    assert not s.query()
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert not any(o.any() for o in others)


def test_refusals(cuda_lib):
    z = torch.zeros(4, 64, device="cuda")
    y = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: cuda_lib.token_logprobs(z.double(), y), lambda: cuda_lib.token_logprobs(z[0], y),
                lambda: cuda_lib.token_logprobs(z.t(), y), lambda: cuda_lib.token_logprobs(z, y.long()),
                lambda: cuda_lib.token_logprobs(z, y[:3]), lambda: cuda_lib.token_logprobs(z.cpu(), None),
                lambda: cuda_lib.token_logprobs_backward(z, torch.zeros(4, device="cuda"), y, None,
                                                         out=torch.zeros(4, 65, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cuda_lib.token_logprobs(z, y, top_k=65), lambda: cuda_lib.token_logprobs(z, y, scale=0.0),
                lambda: cuda_lib.token_logprobs(z, y, scale=float("nan")),
                lambda: cuda_lib.token_logprobs(z.expand(4, 64)[:1].expand(4, 64), y),
                lambda: cuda_lib.token_logprobs_backward(z[:2], torch.zeros(2, device="cuda"), y[:2],
                                                         torch.ones(2, device="cuda"), out=z[1:3])):
        with pytest.raises(cuda_lib.NVFP4Error):
            bad()
