"""Host-side argument checks of the learner operators' entry points, on the CPU: every case is
rejected, or is an empty call, before the library touches a device.  Placeholder addresses
stand in for device buffers and are never dereferenced."""
import ctypes
import math

import pytest

import nvfp4_w4a4_moe_quantize_gb300 as L
from nvfp4_w4a4_moe_quantize_gb300 import build as B

OK, INVALID, UNSUPPORTED = L.Status.OK, L.Status.INVALID_ARG, L.Status.UNSUPPORTED
P, Q = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x900000)
P2, P1 = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10001)
N = ctypes.c_void_p(0)
BF16, F32, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _forward(lib, logits=P, dtype=BF16, T=4, V=100, ld=100, targets=P, scale=1.0, k=3, logprob=P, lse=P, ent=P,
             top=P, ids=P):
    return lib.token_logprobs(logits, dtype, T, V, ld, targets, -100, scale, k, logprob, lse, ent, top, ids, N)


def test_token_logprobs_checks(lib):
    assert _forward(lib, dtype=3) == INVALID
    assert _forward(lib, T=-1) == INVALID
    assert _forward(lib, V=0) == INVALID
    assert _forward(lib, ld=99) == INVALID
    assert _forward(lib, V=(1 << 20) + 1, ld=1 << 21) == UNSUPPORTED
    assert _forward(lib, T=(1 << 24) + 1) == UNSUPPORTED
    for scale in (0.0, -1.0, math.inf, math.nan, 3e38):
        assert _forward(lib, scale=scale) == INVALID
    assert _forward(lib, k=-1) == INVALID
    assert _forward(lib, k=101) == INVALID
    assert _forward(lib, V=1000, ld=1000, k=129) == UNSUPPORTED
    assert _forward(lib, logits=N) == INVALID
    assert _forward(lib, logits=P1) == INVALID
    assert _forward(lib, logits=P2, dtype=F32) == INVALID        # aligned to its element
    assert _forward(lib, lse=N) == INVALID
    assert _forward(lib, logprob=N) == INVALID                   # targets and logprob together
    assert _forward(lib, targets=N) == INVALID
    assert _forward(lib, ids=N) == INVALID
    assert _forward(lib, T=0) == OK


def _backward(lib, logits=P, dtype=BF16, T=4, V=100, ld=100, targets=P, scale=1.0, lse=P, ent=P, dlp=P, dent=P, out=Q,
              ldd=100):
    return lib.token_logprobs_backward(logits, dtype, T, V, ld, targets, -100, scale, lse, ent, dlp, dent, out, ldd, N)


def test_token_logprobs_backward_checks(lib):
    assert _backward(lib, ldd=99) == INVALID
    assert _backward(lib, targets=N) == INVALID                  # dlogprob needs targets
    assert _backward(lib, ent=N) == INVALID                      # dentropy needs entropy
    assert _backward(lib, out=N) == INVALID
    assert _backward(lib, out=P, ldd=128) == INVALID             # in place with another pitch
    assert _backward(lib, out=ctypes.c_void_p(0x10000 + 200)) == INVALID      # overlaps
    assert _backward(lib, scale=math.nan) == INVALID
    assert _backward(lib, lse=N) == INVALID
    assert _backward(lib, T=0) == OK


def test_distill_checks(lib):
    def f(logits=P, dtype=BF16, T=4, V=100, ld=100, ids=P, val=P, K=5, scale=1.0, loss=P, lse=P):
        return lib.distill_topk(logits, dtype, T, V, ld, ids, val, K, 1, scale, loss, lse, N)

    def b(K=5, out=Q, ldd=100, loss=P, T=4, scale=1.0, dloss=P):
        return lib.distill_topk_backward(P, BF16, T, 100, 100, P, P, K, 0, scale, dloss, loss, N, out, ldd, N)

    assert f(K=0) == INVALID and b(K=0) == INVALID
    assert f(K=129) == UNSUPPORTED and b(K=129) == UNSUPPORTED
    assert f(ids=N) == INVALID and f(val=N) == INVALID and f(loss=N) == INVALID
    assert f(dtype=-1) == INVALID and f(V=-5) == INVALID and f(scale=0.0) == INVALID
    assert b(ldd=64) == INVALID and b(out=N) == INVALID and b(loss=N) == INVALID and b(dloss=P2) == INVALID
    assert b(out=ctypes.c_void_p(0x10000 + 16)) == INVALID
    assert f(T=0) == OK and b(T=0) == OK


def test_norm_checks(lib):
    big = 1 << 40

    def fin(x=P, ldx=64, dtype=BF16, T=4, H=64, w=P, eps=1e-6, n=Q, rstd=P):
        return lib.moe_norm_in(x, ldx, dtype, T, H, w, eps, n, rstd, N)

    def fout(ldy=64, gate=N, gate_rows=0, alpha=1.0, nxt=P, n=Q, rr=P, T=4, w=P):
        return lib.moe_norm_out(P, 64, P, ldy, BF16, T, 64, w, gate, gate_rows, alpha, nxt, 1e-6, Q, n, P, rr, N)

    def bin_(dn=P, ld=64, x=P, w=P, dx=Q, dw=P, ws=P, n=big):
        return lib.moe_norm_in_backward(dn, ld, N, 0, x, 64, P, BF16, 4, 64, w, dx, dw, ws, n, N)

    def bout(dr=P, dn=P, r=P, rr=P, gate=N, gate_rows=0, nxt=P, dg=N, dnext=P, ws=P, n=big, lddn=64):
        return lib.moe_norm_out_backward(dr, 64, dn, lddn, r, 64, P, 64, P, rr, BF16, 4, 64, P, gate, gate_rows, 1.0,
                                         nxt, Q, Q, P, dg, dnext, ws, n, N)

    assert fin(dtype=9) == INVALID and fin(T=-1) == INVALID and fin(H=0) == INVALID and fin(ldx=63) == INVALID
    assert fin(eps=0.0) == INVALID and fin(eps=math.nan) == INVALID
    assert fin(H=8193, ldx=9000) == UNSUPPORTED
    assert fin(x=P1) == INVALID and fin(n=N) == INVALID and fin(w=N) == INVALID and fin(rstd=N) == INVALID
    assert fin(T=0) == OK
    assert fout(ldy=60) == INVALID and fout(alpha=math.inf) == INVALID and fout(w=N) == INVALID
    assert fout(gate_rows=2) == INVALID                          # gate rows without a gate
    assert fout(gate=P, gate_rows=3) == INVALID                  # 4 rows do not split into 3
    assert fout(gate=P, gate_rows=-1) == INVALID and fout(gate=P1) == INVALID
    assert fout(n=N) == INVALID and fout(rr=N) == INVALID        # given with next_weight
    assert fout(T=0) == OK
    assert bin_(dn=N) == INVALID and bin_(ld=10) == INVALID and bin_(dw=N) == INVALID and bin_(dx=N) == INVALID
    assert bin_(ws=N) == L.Status.WORKSPACE and bin_(n=100) == L.Status.WORKSPACE
    assert bout(dn=N) == INVALID and bout(r=N) == INVALID and bout(rr=N) == INVALID and bout(dnext=N) == INVALID
    assert bout(dr=N, nxt=N) == INVALID                          # no gradient arrives
    assert bout(gate=P) == INVALID and bout(gate=P, gate_rows=3, dg=P) == INVALID
    assert bout(lddn=3) == INVALID
    assert bout(ws=P2) == L.Status.WORKSPACE and bout(n=0) == L.Status.WORKSPACE


def test_norm_workspace(lib):
    size = lambda T, g, H: lib.nvfp4_workspace_size(L.OP_NORM_BACKWARD, T, g, 0, H, 0)
    assert size(1, 0, 64) == 512                                 # one range of rows, two sums of 64 floats
    assert size(5, 5, 64) == 5 * 512
    assert size(0, 0, 64) == 0 and size(4, 0, 0) == 0
    assert size(1 << 20, 0, 2048) == 304 * 2 * 2048 * 4          # the ranges that the GPU takes at a time
    assert size(1 << 20, 0, 8192) == 152 * 2 * 8192 * 4
