"""Workspace sizes of the router's losses and the head's log probabilities, on the CPU: a workspace for the largest
batch serves every smaller one."""
import math

import pytest

import nvfp4_w4a4_moe_quantize_gb300 as L
from nvfp4_w4a4_moe_quantize_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


ROWS = sorted({*range(1, 700), *(b + d for b in (1024, 2048, 4096, 4864, 8192, 16384, 32768, 65536, 1 << 20) for d in (-1, 0, 1)
                                 if b + d <= 1 << 20), *(round(math.exp(i / 20)) for i in range(130, 277))})


@pytest.mark.parametrize("V,H", [(1, 8), (1000, 64), (8192, 2048), (50021, 1032), (131072, 512), (131072, 2048), (1 << 20, 16384)])
@pytest.mark.parametrize("op", [L.OP_HEAD_LOGPROBS, L.OP_HEAD_LOGPROBS_BACKWARD])
def test_head_sizes_do_not_fall_as_rows_are_added(lib, op, V, H):
    sizes = [lib.nvfp4_workspace_size(op, T, V, 0, H, 0) for T in ROWS]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), [t for t, a, b in zip(ROWS, sizes, sizes[1:]) if a > b][:5]


@pytest.mark.parametrize("E,S", [(8, 1), (128, 1), (128, 40), (1024, 3)])
def test_balance_sizes_do_not_fall_as_rows_are_added(lib, E, S):
    sizes = [lib.nvfp4_workspace_size(L.OP_BALANCE_LOSS, T, S, E, 0, 0) for T in ROWS]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), [t for t, a, b in zip(ROWS, sizes, sizes[1:]) if a > b][:5]


def test_a_piece_of_the_gradient_is_bounded(lib):
    """d of a piece: 2^28 elements, or 8192 tokens of every row where that is more."""
    for T in (100, 8192, 32768, 1 << 20):
        n = lib.nvfp4_workspace_size(L.OP_HEAD_LOGPROBS_BACKWARD, T, 1 << 20, 0, 64, 0)
        assert n <= 2 * max((1 << 28) + 256 * T, 8192 * T) + T * (4 * 128 + 5 * 64 * 4) + (64 << 20), T
