"""What the binding of the learner operators refuses before the library is called, on the CPU: stand-ins
for device tensors, a stand-in for the library that must not be reached."""
import contextlib

import pytest
import torch

import nvfp4_w4a4_moe_quantize_gb300 as L


class Rows:
    """As much of a device tensor as the checks look at."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16, device=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self.device = torch.device("cpu")    # what the results are allocated on

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (*self.shape[1:], 1)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def contiguous(self):
        return self

    def data_ptr(self):
        return 0x10000


class Library:
    def __getattr__(self, name):
        if name == "nvfp4_workspace_size":
            return lambda *a: 16
        raise AssertionError(f"{name} reached")


@pytest.fixture
def current(monkeypatch):
    """The current device, and streams that make theirs current."""
    now = [0]

    @contextlib.contextmanager
    def stream(s):
        before, now[0] = now[0], s.device_index
        yield
        now[0] = before

    monkeypatch.setattr(L, "load", lambda *a: Library())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    return now


class Stream:
    def __init__(self, device_index):
        self.device_index = device_index


def calls(device):
    z = Rows(4, 64, device=device)
    f = Rows(4, dtype=torch.float32, device=device)
    w = Rows(64, dtype=torch.float32, device=device)
    ids, val = Rows(4, 3, dtype=torch.int32, device=device), Rows(4, 3, dtype=torch.float32, device=device)
    y = Rows(4, dtype=torch.int32, device=device)
    return {
        "token_logprobs": lambda **k: L.token_logprobs(z, y, top_k=3, **k),
        "token_logprobs_backward": lambda **k: L.token_logprobs_backward(z, f, y, f, **k),
        "distill_topk": lambda **k: L.distill_topk(z, ids, val, **k),
        "distill_topk_backward": lambda **k: L.distill_topk_backward(z, ids, val, **k),
        "moe_norm_in": lambda **k: L.moe_norm_in(z, w, **k),
        "moe_norm_in_backward": lambda **k: L.moe_norm_in_backward(z, z, f, w, **k),
        "moe_norm_out": lambda **k: L.moe_norm_out(z, z, w, **k),
        "moe_norm_out_backward": lambda **k: L.moe_norm_out_backward(z, z, f, w, **k),
    }


@pytest.mark.parametrize("name", sorted(calls(0)))
def test_rows_of_another_device_are_refused(current, name):
    """The launch, its limits and the status word are the current device's."""
    current[0] = 1
    with pytest.raises(ValueError, match="current"):
        calls(0)[name]()
    with pytest.raises(AssertionError, match="reached"):   # on their own device the rows go through
        calls(1)[name]()


@pytest.mark.parametrize("name", sorted(calls(0)))
def test_a_stream_of_another_device_is_refused(current, name):
    with pytest.raises(ValueError, match="current"):
        calls(0)[name](stream=Stream(1))
    with pytest.raises(AssertionError, match="reached"):
        calls(0)[name](stream=Stream(0))


@pytest.mark.parametrize("index", [2 ** 32, 2 ** 31, -2 ** 31 - 1])
def test_ignore_index_beyond_32_bits_is_refused(current, index):
    """It is compared with int32 targets: cut to 32 bits, 2^32 would ignore token 0."""
    z, y, f = Rows(4, 64), Rows(4, dtype=torch.int32), Rows(4, dtype=torch.float32)
    with pytest.raises(ValueError, match="ignore_index"):
        L.token_logprobs(z, y, ignore_index=index)
    with pytest.raises(ValueError, match="ignore_index"):
        L.token_logprobs_backward(z, f, y, f, ignore_index=index)


@pytest.mark.parametrize("k", [2 ** 32 + 3, -2 ** 32 + 3])
def test_top_k_beyond_32_bits_is_refused(current, k):
    with pytest.raises(ValueError, match="top_k"):
        L.token_logprobs(Rows(0, 64), top_k=k)
