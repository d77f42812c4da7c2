"""GPU parity of the norms around the block (moe_norm_in, moe_norm_out and their backwards) with
the float64 oracle.

Bounds, u = 2^-24.  A row's sum takes 16 terms in a thread, 5 steps in a warp and at most 16
across warps: 40 u with the products' rounding; rstd, of the mean's root, half of that and
3 u: 24 u.  A norm's output has three more roundings: 28 u of itself.  Gradients: the mean of
products is off by 44 u of the mean of their sizes (with rstd's given value exact); sums over T
rows are chains of at most T + 100 steps, of terms with 60 u each.  Outputs of 16 bits
add half a unit in the last place."""
import numpy as np
import pytest
import torch

from oracle import learner as O
from test_gpu_logits import DT, HALF_ULP, TINY, U, f64, near, store

pytestmark = pytest.mark.gpu


def t32(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def as32(a):
    return None if a is None else np.asarray(a, np.float32).astype(np.float64)


def make_gate(kind, T, H, rng):
    if kind == "none":
        return None
    return as32(rng.uniform(-1, 1, T)) if kind == "token" else as32(rng.normal(size=(int(kind), H)))


def half(dtype, ref):
    return HALF_ULP[dtype] * 1.01 * np.abs(ref) + TINY[dtype]


def stored(dtype, ref):
    """The reference as the type can hold it: beyond its largest value (a zero row's rstd is
    1 / sqrt(eps), and its gradient is multiplied by it twice) float16 rounds to infinity."""
    over = 2.0 ** 16 * (1 - 2.0 ** -12) if dtype == torch.float16 else np.inf
    return np.where(np.abs(ref) >= over, np.copysign(np.inf, ref), ref)


def check(lib, T, H, dtype, kind, alpha=1.0, nxt=True, pad=0, lead=0, eps=1e-6, zero_rows=()):
    rng = np.random.default_rng(T * 31 + H + pad)
    dt = DT[dtype]
    xa, ya = rng.normal(0, 2.0, (T, H)), rng.normal(0, 0.3, (T, H))
    for z in zero_rows:
        xa[z] = ya[z] = 0.0
    x, y = store(xa, dtype, pad, lead), store(ya, dtype, pad, lead)
    w, wn = as32(1 + 0.2 * rng.normal(size=H)), as32(1 + 0.2 * rng.normal(size=H))
    gate = make_gate(kind, T, H, rng)
    e32 = float(np.float32(eps))
    a32 = float(np.float32(alpha))
    r, n, ry, rr = lib.moe_norm_out(x, y, t32(w), gate=t32(gate), residual_scale=alpha,
                                    next_weight=t32(wn) if nxt else None, eps=eps)
    xf, yf, rf = f64(x), f64(y), f64(r)
    ref_ry = O.rstd(yf, e32)
    near(ry.cpu(), ref_ry, 24 * U * ref_ry)
    ref = O.norm_out(xf, yf, w, gate, a32, e32)
    near(rf, ref, 30 * U * (np.abs(a32 * xf) + np.abs(ref - a32 * xf)) + half(dt, ref))
    if nxt:
        ref_rr = O.rstd(rf, e32)
        near(rr.cpu(), ref_rr, 24 * U * ref_rr)
        ref_n = rf * ref_rr[:, None] * wn
        near(f64(n), ref_n, 30 * U * np.abs(ref_n) + half(dt, ref_n))
        # the norm alone gives the same bits
        n2, rr2 = lib.moe_norm_in(r, t32(wn), eps=eps)
        assert torch.equal(n, n2) and torch.equal(rr, rr2)
    else:
        assert n is None and rr is None
    # backward, with the kernel's own rstd and r
    dr, dn = store(rng.normal(size=(T, H)), dtype, pad, lead), store(rng.normal(size=(T, H)), dtype, pad, lead)
    got = lib.moe_norm_out_backward(dr, y, ry, t32(w), gate=t32(gate), residual_scale=alpha,
                                    dn=dn if nxt else None, r=r if nxt else None, rstd_r=rr,
                                    next_weight=t32(wn) if nxt else None)
    assert lib.nvfp4_status_check() == 0
    ryf, rrf = f64(ry), f64(rr) if nxt else None
    drf, dnf = f64(dr), f64(dn) if nxt else None
    want = O.norm_out_backward(drf, yf, ryf, w, gate, a32, dnf, rf, rrf, wn)
    d = want[0] / a32
    yhat, g = yf * ryf[:, None], O.gate_rows(gate, T)
    # size of the error in d, in units of u
    ed = 4 * np.abs(d)
    if nxt:
        u1, rhat = dnf * wn, rf * rrf[:, None]
        ed = ed + 8 * rrf[:, None] * np.abs(u1) + 8 * np.abs(drf) + 60 * rrf[:, None] * np.abs(rhat) * np.abs(
            u1 * rhat).mean(1, keepdims=True)
    near(f64(got[0]), stored(dt, want[0]), U * abs(a32) * ed + half(dt, want[0]))
    v, ev = d * g * w, (ed + 4 * np.abs(d)) * np.abs(g * w)
    ey = ryf[:, None] * (ev + 8 * np.abs(v) + np.abs(yhat) * (60 * np.abs(v * yhat) + np.abs(ev * yhat)).mean(1, keepdims=True))
    near(f64(got[1]), stored(dt, want[1]), U * ey + half(dt, want[1]))
    chain = T + 160
    near(got[2].cpu(), want[2], U * ((chain * np.abs(d) + ed) * np.abs(g * yhat)).sum(0) + 1e-37)
    if gate is None:
        assert got[3] is None
    else:
        full = ((chain + 60) * np.abs(d) + ed) * np.abs(w * yhat)
        near(got[3].cpu(), want[3], U * (full.sum(1) if gate.ndim == 1 else full.reshape(len(gate), -1, H).sum(1)) + 1e-37)
    if nxt:
        near(got[4].cpu(), want[4], U * chain * np.abs(dnf * rhat).sum(0) + 1e-37)
        # the norm's own backward, with and without the residual's gradient
        dx, dw = lib.moe_norm_in_backward(dn, r, rr, t32(wn), dresidual=dr)
        near(f64(dx), stored(dt, d), U * ed + half(dt, d))
        near(dw.cpu(), want[4], U * chain * np.abs(dnf * rhat).sum(0) + 1e-37)
        alone, _ = lib.moe_norm_in_backward(dn, r, rr, t32(wn))
        near(f64(alone), stored(dt, d - drf), U * (ed + np.abs(drf)) + half(dt, d - drf))
        only = lib.moe_norm_out_backward(None, y, ry, t32(w), gate=t32(gate), residual_scale=alpha, dn=dn, r=r,
                                         rstd_r=rr, next_weight=t32(wn))
        near(f64(only[0]), stored(dt, a32 * (d - drf)), abs(a32) * U * (ed + np.abs(drf)) + half(dt, a32 * (d - drf)))
    else:
        assert got[4] is None
    return x, y, w, wn, gate, (r, n, ry, rr), got


@pytest.mark.parametrize("T,H", [(1, 1), (1, 2048), (3, 7), (2, 8), (5, 512), (4, 520), (6, 1001), (9, 4096), (3, 8192),
                                 (2, 8191), (1300, 64), (700, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["none", "token"])
def test_norm(cuda_lib, T, H, dtype, kind):
    check(cuda_lib, T, H, dtype, kind, alpha=0.5, nxt=True)


@pytest.mark.parametrize("T,H,kind", [(6, 1001, "3"), (14, 256, "7"), (14, 256, "14"), (1300, 72, "650"), (777, 129, "7"),
                                      (8, 8192, "1")])
@pytest.mark.parametrize("nxt", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_gate_rows(cuda_lib, T, H, kind, nxt, dtype):
    check(cuda_lib, T, H, dtype, kind, alpha=-1.25, nxt=nxt)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H,pad,lead", [(256, 0, 1), (256, 8, 0), (256, 3, 5), (250, 6, 8)])
def test_norm_strides_and_zero_rows(cuda_lib, dtype, H, pad, lead):
    check(cuda_lib, 5, H, dtype, "token", pad=pad, lead=lead, zero_rows=(0, 4), eps=1e-5)


def test_norm_rows_do_not_depend_on_the_batch(cuda_lib):
    x, y, w, wn, gate, out, _ = check(cuda_lib, 1300, 512, "bf16", "token")
    for r in (0, 700, 1299):
        one = cuda_lib.moe_norm_out(x[r:r + 1], y[r:r + 1], t32(w), gate=t32(gate[r:r + 1]), next_weight=t32(wn))
        for a, b in zip(out, one):
            assert torch.equal(a[r:r + 1], b)


def test_norm_gradient_by_differences(cuda_lib):
    rng = np.random.default_rng(3)
    T, H = 12, 300
    x, y = (store(rng.normal(size=(T, H)), "f32") for _ in range(2))
    w, wn, gate = t32(rng.normal(size=H)), t32(rng.normal(size=H)), t32(rng.normal(size=(3, H)))
    cr, cn = t32(rng.normal(size=(T, H))), t32(rng.normal(size=(T, H)))

    def value(x=x, y=y, w=w, gate=gate, wn=wn):
        r, n, _, _ = cuda_lib.moe_norm_out(x, y, w, gate=gate, residual_scale=0.7, next_weight=wn, eps=1e-3)
        return (cr.double() * r + cn.double() * n).sum().item()

    r, _, ry, rr = cuda_lib.moe_norm_out(x, y, w, gate=gate, residual_scale=0.7, next_weight=wn, eps=1e-3)
    dx, dy, dw, dg, dnext = cuda_lib.moe_norm_out_backward(cr, y, ry, w, gate=gate, residual_scale=0.7, dn=cn, r=r,
                                                           rstd_r=rr, next_weight=wn)
    for name, base, grad in (("x", x, dx), ("y", y, dy), ("w", w, dw), ("gate", gate, dg), ("wn", wn, dnext)):
        dirn = t32(rng.normal(size=tuple(base.shape)))
        h = 2.0 ** -9
        num = (value(**{name: base + h * dirn}) - value(**{name: base - h * dirn})) / (2 * h)
        want = (grad.double() * dirn.double()).sum().item()
        # 3600 outputs of size ~1 rounded to float32 add in quadrature: 60 * 4 u / h; third derivatives h^2 of ~1e3
        assert abs(num - want) < 8 * 60 * 4 * U / h + h * h * 1e3, name


def test_empty_batch(cuda_lib):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    r, n, ry, rr = cuda_lib.moe_norm_out(x, x, w, next_weight=w)
    assert r.shape == (0, 64) and n.shape == (0, 64)
    got = cuda_lib.moe_norm_out_backward(x, x, ry, w, dn=x, r=x, rstd_r=rr, next_weight=w)
    assert not got[2].any() and not got[4].any()
    assert not cuda_lib.moe_norm_in_backward(x, x, ry, w)[1].any()


def test_norm_copies_belong_to_the_given_stream(cuda_lib):
    """Dense copies of strided weights, read on the given stream after the call has returned."""
    T, H = 64, 1024
    x = torch.randn(T, H, device="cuda")
    w = torch.rand(H, device="cuda") + 0.5
    w2 = torch.stack((w, w), -1)[..., 0]
    assert not w2.is_contiguous()
    want, rstd = cuda_lib.moe_norm_in(x, w2)
    want_back = cuda_lib.moe_norm_in_backward(x, x, rstd, w2)
    torch.zeros(H, device="cuda")   # every kernel has run once: loading one could wait
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)   # some 50 ms, in which the other stream gets its work done
    got = cuda_lib.moe_norm_in(x, w2, stream=s)[0]
    got_back = cuda_lib.moe_norm_in_backward(x, x, rstd, w2, stream=s)
    others = [torch.zeros(H, device="cuda") for _ in range(64)]
    assert not s.query()
    s.synchronize()
    for a, b in zip((want, *want_back), (got, *got_back)):
        assert torch.equal(a, b)
    assert not any(o.any() for o in others)


def test_norm_refusals(cuda_lib):
    x = torch.zeros(6, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    f = lambda *s: torch.ones(*s, device="cuda")
    for bad in (lambda: cuda_lib.moe_norm_in(x, w.bfloat16()), lambda: cuda_lib.moe_norm_in(x, f(63)),
                lambda: cuda_lib.moe_norm_out(x, x[:5], w), lambda: cuda_lib.moe_norm_out(x, x.float(), w),
                lambda: cuda_lib.moe_norm_out(x, x, w, gate=f(5)), lambda: cuda_lib.moe_norm_out(x, x, w, gate=f(2, 63)),
                lambda: cuda_lib.moe_norm_out_backward(None, x, f(6), w),
                lambda: cuda_lib.moe_norm_out_backward(x, x, f(6), w, dn=x)):
        with pytest.raises(ValueError):
            bad()
    wide = torch.zeros(2, 8200, device="cuda")
    for bad in (lambda: cuda_lib.moe_norm_out(x, x, w, gate=f(4, 64)), lambda: cuda_lib.moe_norm_in(x, w, eps=0.0),
                lambda: cuda_lib.moe_norm_in(wide, f(8200)),
                lambda: cuda_lib.moe_norm_in_backward(x, x, f(6), w, workspace=torch.empty(16, dtype=torch.uint8,
                                                                                          device="cuda"))):
        with pytest.raises(cuda_lib.NVFP4Error):
            bad()


@pytest.mark.parametrize("shape", [(0, 64), (), (1, 6, 64)])
def test_norm_gate_without_rows_is_refused(cuda_lib, shape):
    x = torch.ones(6, 64, device="cuda")
    w, gate = torch.ones(64, device="cuda"), torch.ones(shape, device="cuda")
    with pytest.raises(ValueError):
        cuda_lib.moe_norm_out(x, x, w, gate=gate)
    with pytest.raises(ValueError):
        cuda_lib.moe_norm_out_backward(x, x, torch.ones(6, device="cuda"), w, gate=gate)


def test_norm_workspace_is_checked(cuda_lib):
    """Only host-side refusals: memory of the host, another type's elements, bytes apart."""
    x, w = torch.ones(6, 64, device="cuda"), torch.ones(64, device="cuda")
    n = cuda_lib.load().nvfp4_workspace_size(cuda_lib.OP_NORM_BACKWARD, 6, 0, 0, 64, 0)
    rstd = torch.ones(6, device="cuda")
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(n, device="cuda"),
                torch.empty(n, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError):
            cuda_lib.moe_norm_in_backward(x, x, rstd, w, workspace=bad)
        with pytest.raises(ValueError):
            cuda_lib.moe_norm_out_backward(x, x, rstd, w, workspace=bad)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for a, b in zip(cuda_lib.moe_norm_in_backward(x, x, rstd, w, workspace=ws),
                    cuda_lib.moe_norm_in_backward(x, x, rstd, w)):
        assert torch.equal(a, b)
