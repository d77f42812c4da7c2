"""The router's losses where calls are easily refused or answered wrongly."""
import os
import subprocess
import sys

import pytest

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
