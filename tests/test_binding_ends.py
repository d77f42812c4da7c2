"""What the binding of the router's losses and the head's log probabilities refuses before the library is called,
on the CPU: stand-ins for device tensors, a stand-in for the library that must not be reached."""
import pytest
import torch

import nvfp4_w4a4_moe_quantize_gb300 as L
from test_binding_rows import Rows, Stream, current  # noqa: F401

F32, I32 = torch.float32, torch.int32


def calls(d):
    x, w, y, f = Rows(4, 64, device=d), Rows(100, 64, device=d), Rows(4, dtype=I32, device=d), Rows(4, dtype=F32, device=d)
    z, ids = Rows(4, 8, dtype=F32, device=d), Rows(4, 2, dtype=I32, device=d)
    dw, one = Rows(4, 2, dtype=F32, device=d), Rows(1, dtype=F32, device=d)
    c, n = Rows(1, 8, dtype=I32, device=d), Rows(1, dtype=I32, device=d)
    return {
        "head_logprobs": lambda **k: L.head_logprobs(x, w, y, **k),
        "head_logprobs_backward": lambda **k: L.head_logprobs_backward(x, w, f, y, f, f, f, **k),
        "moe_balance_loss": lambda **k: L.moe_balance_loss(z, ids, **k),
        "moe_router_backward": lambda **k: L.moe_router_backward(z, ids, dw, True, one, c, n, **k),
    }


@pytest.mark.parametrize("name", sorted(calls(0)))
def test_rows_and_streams_of_another_device_are_refused(current, name):  # noqa: F811
    with pytest.raises(ValueError, match="current"):
        calls(1)[name]()
    with pytest.raises(ValueError, match="current"):
        calls(0)[name](stream=Stream(1))
    with pytest.raises(AssertionError, match="reached"):
        calls(0)[name](stream=Stream(0))


def test_companions_of_another_shape_type_or_device_are_refused(current):  # noqa: F811
    x, w, y, f = Rows(4, 64), Rows(100, 64), Rows(4, dtype=I32), Rows(4, dtype=F32)
    z, ids = Rows(4, 8, dtype=F32), Rows(4, 2, dtype=I32)
    c, n, one = Rows(1, 8, dtype=I32), Rows(1, dtype=I32), Rows(1, dtype=F32)
    bad = [
        lambda: L.head_logprobs(x, Rows(100, 72), y),
        lambda: L.head_logprobs(x, Rows(100, 64, dtype=torch.float16), y),
        lambda: L.head_logprobs(x, w, Rows(5, dtype=I32)),
        lambda: L.head_logprobs(x, w, Rows(4, dtype=torch.int64)),
        lambda: L.head_logprobs(x, w, Rows(4, dtype=I32, device=1)),
        lambda: L.head_logprobs(x, w, y, ignore_index=2 ** 31),
        lambda: L.head_logprobs(Rows(4, 4, 64), w, y),
        lambda: L.head_logprobs_backward(x, w, Rows(3, dtype=F32), y, f),
        lambda: L.head_logprobs_backward(x, w, f, y, Rows(4, dtype=torch.bfloat16)),
        lambda: L.head_logprobs_backward(x, w, f, y, f, ignore_index=-2 ** 31 - 1),
        lambda: L.head_logprobs(x, w, y, workspace=Rows(64, dtype=F32)),
        lambda: L.moe_balance_loss(z, Rows(4, dtype=I32)),
        lambda: L.moe_balance_loss(z, Rows(5, 2, dtype=I32)),
        lambda: L.moe_balance_loss(z, Rows(4, 2, dtype=torch.int64)),
        lambda: L.moe_balance_loss(Rows(4, 8, dtype=torch.float64), ids),
        lambda: L.moe_balance_loss(z, ids, sequences=Rows(1, dtype=I32)),
        lambda: L.moe_balance_loss(z, ids, sequences=Rows(3, dtype=torch.int64)),
        lambda: L.moe_balance_loss(z, ids, valid=Rows(3, dtype=torch.bool)),
        lambda: L.moe_balance_loss(z, ids, valid=Rows(4, dtype=F32)),
        lambda: L.moe_router_backward(z, ids, Rows(4, 3, dtype=F32)),
        lambda: L.moe_router_backward(z, ids, dloss=one),
        lambda: L.moe_router_backward(z, ids, dloss=one, counts=c),
        lambda: L.moe_router_backward(z, ids, dloss=Rows(2, dtype=F32), counts=c, tokens=n),
        lambda: L.moe_router_backward(z, ids, dloss=one, counts=Rows(8, dtype=I32), tokens=n),
        lambda: L.moe_router_backward(z, ids, Rows(4, 2, dtype=F32), out=Rows(4, 9, dtype=F32)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
