"""Host-side argument checks of the router's losses and the head's log probabilities, on the CPU: every case is
rejected, or is an empty call, before the library touches a device.  Placeholder addresses stand in for device
buffers and are never dereferenced."""
import ctypes
import math

import pytest

import nvfp4_w4a4_moe_quantize_gb300 as L
from nvfp4_w4a4_moe_quantize_gb300 import build as B

OK, INVALID, UNSUPPORTED, WORKSPACE = L.Status.OK, L.Status.INVALID_ARG, L.Status.UNSUPPORTED, L.Status.WORKSPACE
N = ctypes.c_void_p(0)
BF16, F32, F16 = 0, 1, 2


def at(a):
    return ctypes.c_void_p(a)


P, Q, R, S = at(0x100000), at(0x2000000), at(0x4000000), at(0x6000000)
WS = at(0x80000000)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _forward(lib, x=P, ldx=64, w=Q, ldw=64, dtype=BF16, T=4, V=100, H=64, y=R, scale=1.0, lp=R, lse=R, ent=R, ws=WS, n=BIG):
    return lib.head_logprobs(x, ldx, w, ldw, dtype, T, V, H, y, -100, scale, lp, lse, ent, ws, n, N)


def test_head_logprobs_checks(lib):
    for bad in (dict(dtype=3), dict(T=-1), dict(V=0), dict(H=0), dict(ldx=56), dict(ldw=56)):
        assert _forward(lib, **bad) == INVALID, bad
    for scale in (0.0, -1.0, math.inf, math.nan, 3e38):
        assert _forward(lib, scale=scale) == INVALID
    for bad in (dict(dtype=F32), dict(V=(1 << 20) + 1), dict(T=(1 << 20) + 1), dict(H=16392, ldx=16392, ldw=16392),
                dict(H=63), dict(H=60), dict(ldx=68), dict(ldw=66), dict(ldx=1 << 33)):
        assert _forward(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(x=N), dict(w=N), dict(x=at(0x100008)), dict(w=at(0x2000002)), dict(lse=N), dict(lse=at(0x4000002)),
                dict(lp=N), dict(y=N), dict(y=at(0x4000001)), dict(ent=at(0x4000001))):
        assert _forward(lib, **bad) == INVALID, bad
    need = lib.nvfp4_workspace_size(L.OP_HEAD_LOGPROBS, 4, 100, 0, 64, 0)
    assert need > 0
    for bad in (dict(ws=N), dict(ws=at(0x80000008)), dict(n=need - 1)):
        assert _forward(lib, **bad) == WORKSPACE, bad
    assert _forward(lib, T=0, x=N, ws=N, n=0) == OK


def _backward(lib, x=P, ldx=64, w=Q, ldw=64, dtype=BF16, T=4, V=100, H=64, y=R, lse=R, ent=R, g=R, h=R, dx=S, dw=at(0x7000000),
              scale=1.0, ws=WS, n=BIG):
    return lib.head_logprobs_backward(x, ldx, w, ldw, dtype, T, V, H, y, -100, scale, lse, ent, g, h, dx, dw, ws, n, N)


def test_head_logprobs_backward_checks(lib):
    assert _backward(lib, dtype=F32) == UNSUPPORTED
    assert _backward(lib, H=65, ldx=72, ldw=72) == UNSUPPORTED
    assert _backward(lib, scale=math.nan) == INVALID
    for bad in (dict(dx=N, dw=N), dict(y=N), dict(ent=N), dict(lse=N), dict(dx=at(0x6000008)), dict(dw=at(0x7000002)),
                dict(g=at(0x4000002)), dict(h=at(0x4000001))):
        assert _backward(lib, **bad) == INVALID, bad
    # outputs on the inputs, or on one another
    for bad in (dict(dx=P), dict(dx=at(0x100000 + 496)), dict(dw=Q), dict(dw=at(0x2000000 - 16)), dict(dx=Q), dict(dw=P),
                dict(dw=S), dict(dw=at(0x6000000 + 496))):
        assert _backward(lib, **bad) == INVALID, bad
    need = lib.nvfp4_workspace_size(L.OP_HEAD_LOGPROBS_BACKWARD, 4, 100, 0, 64, 0)
    assert _backward(lib, n=need - 1) == WORKSPACE
    assert _backward(lib, ws=at(0x80000004)) == WORKSPACE
    assert _backward(lib, T=0, dw=N, x=N, ws=N, n=0) == OK


def test_head_workspaces_hold_pieces_not_logits(lib):
    """The forward keeps 12 bytes of every row and 128 tokens, the backward a piece of d: far from a copy of the
    logits where there are many rows, and linear in them."""
    f = lambda T: lib.nvfp4_workspace_size(L.OP_HEAD_LOGPROBS, T, 131072, 0, 2048, 0)  # noqa: E731
    b = lambda T: lib.nvfp4_workspace_size(L.OP_HEAD_LOGPROBS_BACKWARD, T, 131072, 0, 2048, 0)  # noqa: E731
    for T in (8192, 65536):
        assert f(T) < T * 131072 * 2 // 10
        assert b(T) < T * 131072 * 2 // 2
    assert 7.9 < f(65536) / f(8192) < 8.1
    for size in (f, b):
        assert size(0) == 0 and size(-1) == 0 and size(1) > 0


def _loss(lib, z=P, dtype=F32, T=64, E=8, ld=8, ids=R, k=2, seq=N, nseq=1, valid=N, loss=R, counts=R, sums=R, tokens=R, ws=WS, n=BIG):
    return lib.moe_balance_loss(z, dtype, T, E, ld, ids, k, seq, nseq, valid, loss, counts, sums, tokens, ws, n, N)


def test_balance_loss_checks(lib):
    for bad in (dict(dtype=3), dict(T=-1), dict(E=0), dict(ld=7), dict(k=0), dict(k=9), dict(nseq=0), dict(nseq=2),
                dict(seq=at(0x4000002), nseq=2), dict(z=N), dict(z=at(0x100002)), dict(ids=N), dict(ids=at(0x4000001)),
                dict(loss=N), dict(counts=N), dict(sums=N), dict(tokens=N), dict(loss=at(0x4000002))):
        assert _loss(lib, **bad) == INVALID, bad
    for bad in (dict(E=1025, ld=1025), dict(E=64, ld=64, k=33), dict(T=(1 << 24) + 1), dict(seq=R, nseq=(1 << 20) + 1)):
        assert _loss(lib, **bad) == UNSUPPORTED, bad
    assert _loss(lib, T=5000, n=16) == WORKSPACE
    assert _loss(lib, T=5000, ws=N) == WORKSPACE
    assert _loss(lib, seq=R, nseq=3, ws=N) == WORKSPACE
    assert lib.nvfp4_workspace_size(L.OP_BALANCE_LOSS, 64, 1, 8, 0, 0) == 0     # few rows need none


def _router(lib, z=P, dtype=F32, T=64, E=8, ld=8, ids=R, k=2, dw=R, dloss=R, counts=R, tokens=R, seq=N, nseq=1, valid=N, out=Q,
            ldd=8):
    return lib.moe_router_backward(z, dtype, T, E, ld, ids, k, dw, 1, dloss, counts, tokens, seq, nseq, valid, out, ldd, N)


def test_router_backward_checks(lib):
    for bad in (dict(dtype=5), dict(ldd=7), dict(dw=N, dloss=N), dict(ids=N), dict(counts=N), dict(tokens=N), dict(out=N),
                dict(dw=at(0x4000002)), dict(out=P, ldd=16), dict(out=at(0x100000 + 64)), dict(nseq=4), dict(k=9)):
        assert _router(lib, **bad) == INVALID, bad
    assert _router(lib, E=2000, ld=2000, ldd=2000) == UNSUPPORTED
    assert _router(lib, T=0, z=N, out=N, dw=N, dloss=N) == OK
