"""The router's losses where calls are easily answered wrongly: numbers of experts next to the limits of a launch,
padding that holds anything, lists of sequences that descend."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import ends as O
from test_gpu_router_loss import check_gradient, check_loss, f64, router

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_any_number_of_experts_as_a_process_s_first_call():
    """Just below 48 KB of dynamic shared memory (E = 372) the static part counts as well; a process that has had a
    larger number before does not show it."""
    code = """
import torch
import nvfp4_w4a4_moe_quantize_gb300 as lib
for E in range(365, 376):
    for T in (8, 500):
        z = torch.arange(T * E, device="cuda").view(T, E).remainder(7).float()
        loss, counts, sums, tokens = lib.moe_balance_loss(z, torch.zeros(T, 1, dtype=torch.int32, device="cuda"))
        want = torch.softmax(z.double(), 1).sum(0)
        assert counts[0, 0] == T and counts.sum() == T and tokens[0] == T
        assert torch.allclose(sums[0].double(), want, rtol=1e-4)
        assert torch.allclose(loss[0].double(), E / T * want[0], rtol=1e-4)
assert lib.nvfp4_status_check() == 0
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("E,k", [(20, 3), (128, 8), (300, 6), (1024, 4)])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_padding_may_hold_anything_in_the_balance_loss_s_gradient(cuda_lib, E, k, dtype):
    """Tokens of no sequence and padding tokens hold NaN and infinity: their gradient is 0, the others' as ever."""
    T = 203
    zt, ids, it, rng = router(T, E, k, E, dtype)
    cuts, valid = np.array([5, 60, 60, 61, 190], np.int32), rng.random(T) < 0.7
    out = np.ones(T, bool)
    out[5:190] = ~valid[5:190]
    zz = np.where(out[:, None], 0.0, f64(zt))
    bad = torch.from_numpy(out).cuda()
    zt[bad] = torch.where(torch.arange(E, device="cuda") % 2 == 0, float("nan"), float("inf")).to(zt.dtype)
    _, counts, _, tokens, st, vt = check_loss(cuda_lib, zz, ids, zt, it, cuts, valid)
    got = check_gradient(cuda_lib, zz, ids, zt, it, dtype, dloss=rng.normal(size=4), parts=(counts, tokens, st, vt),
                         sequences=cuts, valid=valid)
    assert (got[bad] == 0).all()


@pytest.mark.parametrize("T,cuts", [(5000, [0, 4000, 100, 5000]), (96, [0, 96, 0, 96]), (5000, [4000, 5000, 0, 700]),
                                    (5000, [0, 5000] * 40), (20, [0, 20, 0, 20, 3, 9]), (20, [19, 20, 0, 7]),
                                    (5000, [0, 10, 5001, 5002]), (5000, [-7, 10, 40, 4999])])
def test_results_of_lists_that_are_not_in_order(cuda_lib, T, cuts):
    """The status is set.  A pair that descends or leaves the batch has the loss and sums NaN and nothing counted; a
    proper one its own results, or the same where the list descends: never other numbers, whatever the workspace held."""
    zt, ids, it, _ = router(T, 16, 2, 9)
    S, st = len(cuts) - 1, torch.tensor(cuts, dtype=torch.int32, device="cuda")
    n = cuda_lib.load().nvfp4_workspace_size(cuda_lib.OP_BALANCE_LOSS, T, S, 16, 0, 0)
    bad = np.array([a < 0 or b < a or b > T for a, b in zip(cuts[:-1], cuts[1:])])
    descends = any(b < a for a, b in zip(cuts[:-1], cuts[1:]))
    want = O.balance_loss(f64(zt), ids, [min(max(c, 0), T) for c in cuts])
    for fill in (0, 1, 255):
        ws = torch.full((max(n, 16),), fill, dtype=torch.uint8, device="cuda")
        loss, counts, sums, tokens = cuda_lib.moe_balance_loss(zt, it, sequences=st, workspace=ws)
        assert cuda_lib.nvfp4_status_check() == cuda_lib.Status.DEVICE_STATUS
        nan = torch.isnan(loss).cpu().numpy()
        assert nan[bad].all() and (descends or (nan == bad).all())
        for s in range(S):
            if nan[s]:
                assert torch.isnan(sums[s]).all() and (counts[s] == 0).all() and tokens[s] == 0
            else:
                assert np.array_equal(counts[s].cpu().numpy(), want[1][s]) and tokens[s] == want[3][s]
                assert np.allclose(f64(sums[s]), want[2][s], rtol=1e-5) and np.isclose(loss[s].item(), want[0][s], rtol=1e-5)


@pytest.mark.parametrize("T", [20, 5000])
@pytest.mark.parametrize("cuts", [[9, 3], [-1, 9], [0, 5001]])
def test_a_single_sequence_out_of_range_counts_nothing(cuda_lib, T, cuts):
    """The same answer from a few rows and from many."""
    zt, _, it, _ = router(T, 8, 2, 3)
    loss, counts, sums, tokens = cuda_lib.moe_balance_loss(zt, it, sequences=torch.tensor(cuts, dtype=torch.int32, device="cuda"))
    assert cuda_lib.nvfp4_status_check() == cuda_lib.Status.DEVICE_STATUS
    assert torch.isnan(loss).all() and torch.isnan(sums).all() and (counts == 0).all() and (tokens == 0).all()
