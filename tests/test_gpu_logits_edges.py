"""Operators on rows of logits at the places where a row is cut: ends of slices, parts of a row in
several CTAs, rows that follow one another in a cluster.  Bounds as in test_gpu_logits."""
import numpy as np
import pytest
import torch

from oracle import learner as O
from test_gpu_logits import U, check_backward, check_distill, check_forward, eps, f64, logits, near, store, teacher

pytestmark = pytest.mark.gpu


def slice_ends(V, width=4):
    """The first and last `width` tokens of every slice of a row."""
    slices = 8 if V >= 65536 else 4 if V >= 32768 else 2 if V >= 16384 else 1
    chunks = -(-V // 8)
    per = -(-chunks // slices)
    out = []
    for s in range(slices):
        lo, hi = min(V, 8 * s * per), min(V, 8 * (s + 1) * per)
        out += [*range(lo, lo + width), *range(hi - width, hi)]
    return np.unique(out)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [9003, 40005, 70001])
def test_listed_tokens_at_the_ends_of_a_slice(cuda_lib, tail, dtype, V):
    """A row's ends, which do not arrive in whole 16-byte words, hold listed tokens: at every
    alignment the row gives what it gives aligned."""
    T = 6
    z, rng = logits(T, V, V)
    ends = slice_ends(V)
    z[:, ends] = rng.normal(4.0, 2.0, (T, ends.size))   # mass that would be missed in the tail's sum
    ids = np.stack([rng.permutation(ends) for _ in range(T)]).astype(np.int32)
    _, val = teacher(T, V, ends.size, rng)
    w = rng.normal(size=T)
    want_loss, want = check_distill(cuda_lib, store(z, dtype), ids, val, tail, w=w)
    it, vt = torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda()
    wt = torch.from_numpy(w.astype(np.float32)).cuda()
    for lead in range(1, 8):
        for pad in (0, 8):
            loss, d = cuda_lib.distill_topk_backward(store(z, dtype, pad, lead), it, vt, wt, tail)
            assert torch.equal(loss, want_loss) and torch.equal(d, want)
    assert cuda_lib.nvfp4_status_check() == 0


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,V,T", [("bf16", 131072, 1300), ("f32", 70001, 640), ("f16", 33001, 200)])
def test_rows_of_a_cluster_exchange_their_own_sums(cuda_lib, tail, dtype, V, T):
    """Neighbouring rows whose slices' maxima differ by tens, over several CTAs: every row of a long
    batch gives what it gives alone, so no CTA took another row's message for its own."""
    n, K = 8, 24
    z, rng = logits(n, V, V)
    z += 15.0 * (-1.0) ** np.arange(n)[:, None]                        # neighbours differ by 30,
    z += np.repeat(rng.normal(0, 10.0, (n, 64)), -(-V // 64), 1)[:, :V]   # and a row's slices by tens
    ids, val = teacher(n, V, K, rng)
    it, vt, zt = torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda(), store(z, dtype)
    one = [cuda_lib.distill_topk_backward(zt[r:r + 1], it[r:r + 1], vt[r:r + 1], None, tail) for r in range(n)]
    few_loss, few = torch.cat([o[0] for o in one]), torch.cat([o[1] for o in one])
    check_distill(cuda_lib, zt, ids, val, tail)
    pick = torch.arange(T, device="cuda") % n
    for _ in range(3):
        loss, d = cuda_lib.distill_topk_backward(zt[pick], it[pick], vt[pick], None, tail)
        assert torch.equal(loss, few_loss[pick]) and torch.equal(d, few[pick])
    assert cuda_lib.nvfp4_status_check() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,K", [(5, 3), (1003, 20), (33001, 100), (131072, 64)])
def test_distill_masses_that_do_not_add_up_to_one(cuda_lib, dtype, V, K):
    """With the tail: the list alone is allowed and holds 0.8 or 1.3; it holds 1.3 in an open row; it
    holds 1.3 and one of its tokens is excluded by the student without having mass.  check_distill's
    bound takes p twice over, which covers 1.3 p with the rounding of 1.3, (K / 8 + 16) u."""
    z, rng = logits(4, V, V + K)
    ids, val = teacher(4, V, K, rng)
    for r in (0, 1):
        keep = z[r, ids[r]].copy()
        z[r] = -np.inf
        z[r, ids[r]] = np.where(np.isfinite(keep), keep, 0.0)
    val[1:] += np.float32(np.log(1.3 / 0.8))
    val[3, 1] = -np.inf
    z[3, ids[3, 1]] = -np.inf
    zt = store(z, dtype)
    w = np.array([1.0, -0.5, 2.0, 1.0])
    _, d = check_distill(cuda_lib, zt, ids, val, True, 1.3, w)
    if dtype == "f32":   # the loss does not change with a shift of the row
        assert (d.double().sum(1).abs() < 1e-4).all()


def test_distill_gradient_by_differences_where_the_masses_do_not_add_up(cuda_lib):
    """As test_gradient_by_differences, for lists of more than one and rows of the list alone."""
    V, K = 2003, 40
    z, rng = logits(6, V, 8)
    ids, val = teacher(6, V, K, rng)
    val[3:] += np.float32(np.log(1.4 / 0.8))
    for r in (0, 1, 5):
        keep = z[r, ids[r]].copy()
        z[r] = -np.inf
        z[r, ids[r]] = keep
    zt, it, vt = store(z, "f32"), torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda()
    w = torch.rand(6, generator=torch.Generator().manual_seed(1)).cuda()
    _, d = cuda_lib.distill_topk_backward(zt, it, vt, w)
    step = 2.0 ** -5
    for seed in range(3):
        dirn = torch.randn(zt.shape, generator=torch.Generator().manual_seed(10 + seed)).cuda()
        lo = lambda x: (w * cuda_lib.distill_topk(x, it, vt)[0]).double().sum().item()
        num = (lo(zt + step * dirn) - lo(zt - step * dirn)) / (2 * step)
        assert abs(num - (d.double() * dirn.double()).sum().item()) < 6 * 4e-6 / step + step ** 2 * 10


@pytest.mark.parametrize("h,scale", [(1e10, 1.0), (1e8, 1e3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_entropy_gradient_of_large_weight_at_excluded_tokens(cuda_lib, h, scale, dtype):
    """Excluded tokens have no gradient however large its weight is."""
    z, rng = logits(5, 6007, 23, masked=0.4)
    zt = store(z, dtype)
    y = rng.integers(0, 6007, 5).astype(np.int32)
    d = check_backward(cuda_lib, zt, y, rng.normal(size=5), h * (1.0 + rng.random(5)), scale)
    assert torch.isfinite(d).all() and not d[torch.isneginf(zt)].any() and d.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [3001, 40009])
def test_entropy_of_rows_with_a_huge_maximum(cuda_lib, dtype, V):
    """A maximum near the type's largest value: the others' distance from it is beyond float32, their
    probability and their part of the entropy are zero."""
    z, rng = logits(4, V, V, masked=0.2)
    y = rng.integers(0, V, 4).astype(np.int32)
    z[np.arange(4), y] = [3.3e38, 2.5e38, 1e38, 1e33]
    got, ref = check_forward(cuda_lib, store(z, dtype), y, 1.0, 0)
    assert (got[2] == 0).all() and (got[0] == 0).all() and (ref["entropy"] == 0).all()


@pytest.mark.parametrize("scale", [0.70948, 1.0, 1.4443842, 1.4487727])
def test_backward_of_rows_far_from_zero(cuda_lib, scale):
    """A probability recomputed from lse carries lse's own rounding and no other of that size: u |lse|
    relatively, beside what rows near zero have (eps, 84 u, 4 u |ln p|)."""
    T, V = 256, 1003
    z, rng = logits(T, V, 77)
    z += (np.exp(rng.uniform(np.log(1e4), np.log(1e6), T)) * rng.choice([-1.0, 1.0], T))[:, None]
    zt = store(z, "f32")
    y = torch.from_numpy(rng.integers(0, V, T).astype(np.int32)).cuda()
    g = np.float32(rng.normal(size=T)).astype(np.float64)
    _, lse, _, _, _ = cuda_lib.token_logprobs(zt, y, scale=scale)
    got = f64(cuda_lib.token_logprobs_backward(zt, lse, y, torch.from_numpy(g.astype(np.float32)).cuda(), scale=scale))
    s = float(np.float32(scale))
    lp, p, l = O.softmax_stats(f64(zt) * s)
    ref = O.token_logprobs_backward(f64(zt), y.cpu().numpy(), g, None, s)
    rel = np.expm1(eps(V) + U * np.abs(l)[:, None] + 84 * U + 4 * U * np.abs(lp))
    near(got, ref, s * np.abs(g)[:, None] * p * rel + 4 * U * np.abs(ref) + 1e-37)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_backward_of_rows_that_an_additive_mask_leaves_empty(cuda_lib, dtype, scale):
    """A mask that adds -1e9 to every token: lse lies where float32 is 64 apart and tells nothing of p; the
    row has nothing to learn from."""
    z, rng = logits(4, 4001, 3)
    z[1] -= 1e9
    z[2] -= 3e7
    z[3, 100:] -= 1e9
    zt = store(z, dtype)
    y = torch.zeros(4, dtype=torch.int32, device="cuda")
    one = torch.ones(4, device="cuda")
    _, lse, ent, _, _ = cuda_lib.token_logprobs(zt, y, scale=scale)
    d = cuda_lib.token_logprobs_backward(zt, lse, y, one, entropy=ent, dentropy=one, scale=scale)
    assert torch.isfinite(d).all() and not d[1:3].any()
    assert d[0].any() and d[3, :100].any() and not d[3, 100:].any()


@pytest.mark.parametrize("T", [2, 640])
def test_a_few_more_threads_than_alternatives(cuda_lib, T):
    """1100 allowed neighbours are 138 threads' chunks: hardly more than the list is long, with many more
    candidates."""
    V = 40000
    rng = np.random.default_rng(T)
    z = np.full((T, V), -np.inf)
    z[:, 8005:9105] = rng.normal(0.0, 1.0, (T, 1100))
    check_forward(cuda_lib, store(z, "f32"), np.full(T, 8500, np.int32), 1.0, 128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(200, 131072), (400, 131072), (200, 70001), (400, 70001), (200, 33001), (330, 20011)])
def test_several_slices_a_cta_of_a_cluster(cuda_lib, dtype, T, V):
    """Between a CTA a slice and a CTA a row: every row gives what it gives alone."""
    n = 8
    z, rng = logits(n, V, V + 1)
    y = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).cuda()
    ids, val = teacher(n, V, 30, rng)
    it, vt, zt = torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda(), store(z, dtype)
    pick = torch.from_numpy(rng.integers(0, n, T)).cuda()
    many = zt[pick]
    for k in (0, 20, 128):
        alone = [cuda_lib.token_logprobs(zt[r:r + 1], y[r:r + 1], top_k=k) for r in range(n)]
        got = cuda_lib.token_logprobs(many, y[pick], top_k=k)
        for i, a in enumerate(got):
            assert a is None or torch.equal(a, torch.cat([o[i] for o in alone])[pick])
    check_forward(cuda_lib, zt, y.cpu().numpy(), 1.0, 128)
    for tail in (False, True):
        alone = [cuda_lib.distill_topk(zt[r:r + 1], it[r:r + 1], vt[r:r + 1], tail) for r in range(n)]
        for i, a in enumerate(cuda_lib.distill_topk(many, it[pick], vt[pick], tail)):
            assert torch.equal(a, torch.cat([o[i] for o in alone])[pick])


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_distill_loss_at_the_lowest_values_is_finite(cuda_lib, tail, dtype):
    """The type's lowest value is a value like any other: where the loss is one that float32 holds, it is not
    infinite.  Listed tokens at the lowest value, with masses that add up to 1.3 (and 0.9); the
    unlisted ones there.  One product of the loss exceeds all others; it carries the roundings of q,
    scale and the sums, 16 u and u a listed token."""
    low = float(torch.finfo({"bf16": torch.bfloat16, "f32": torch.float32}[dtype]).min)
    z, _ = logits(3, 3001, 6)
    z[0, :20] = z[1, :20] = low
    z[2, :] = low
    z[2, :20] = 0.5
    q = np.full((3, 20), 1.0 / 20) * np.array([[1.3], [0.9], [0.7]])
    ids = torch.arange(20, dtype=torch.int32, device="cuda").repeat(3, 1)
    val = torch.from_numpy(np.log(q).astype(np.float32)).cuda()
    for scale in (0.05, 0.7):
        s = float(np.float32(scale))
        mass = np.array([1.3, 0.9, 0.3]) if tail else np.array([1.0, 1.0, 0.0])
        want = -s * low * mass
        zt = store(z, dtype)
        loss = cuda_lib.distill_topk(zt, ids, val, tail, scale)[0]
        both, d = cuda_lib.distill_topk_backward(zt, ids, val, None, tail, scale)
        ok = want < 3e38
        near(f64(loss)[ok], want[ok], 40 * U * want[ok] + 100.0)
        assert torch.equal(loss, both) and torch.isfinite(d).all()
