"""Norms around the block on batches that give every group of threads several rows: the ring of rows in
shared memory is refilled and wraps.  Bounds as in test_gpu_norm."""
import pytest
import torch

from test_gpu_norm import check, t32

pytestmark = pytest.mark.gpu


# (6000 rows of 2048 are 5 a group forward and 10 backward, 12000 of 64 are 3 and 5, 1300 of 8192 are 5 and 9;
# none of the batches is a multiple of the groups)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,kind,nxt", [(6000, 2048, "token", True), (6000, 2048, "none", False), (12000, 64, "token", True),
                                          (1300, 8192, "4", True), (1300, 8192, "token", False), (5001, 520, "3", True),
                                          (3001, 1001, "token", True)])
def test_several_rows_a_group(cuda_lib, T, H, kind, nxt, dtype):
    x, y, w, wn, gate, out, _ = check(cuda_lib, T, H, dtype, kind, alpha=0.5, nxt=nxt)
    for r in (0, 1217, T - 1):   # and the row's bits are those of the row alone
        g = None if gate is None else t32(gate[r:r + 1] if gate.ndim == 1 else gate[r * len(gate) // T:][:1])
        one = cuda_lib.moe_norm_out(x[r:r + 1], y[r:r + 1], t32(w), gate=g, residual_scale=0.5,
                                    next_weight=t32(wn) if nxt else None)
        for a, b in zip(out, one):
            assert a is None or torch.equal(a[r:r + 1], b)


@pytest.mark.parametrize("T,H", [(1, 2048), (777, 1001), (6000, 512)])
def test_norms_in_a_graph(cuda_lib, T, H):
    """Forward and both backwards replayed with new inputs equal the eager calls."""
    g = torch.Generator(device="cuda").manual_seed(T)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, y, dr, dn = (new(T, H).bfloat16() for _ in range(4))
    w, wn, gate = new(H), new(H), new(T)

    def step():
        r, n, ry, rr = cuda_lib.moe_norm_out(x, y, w, gate=gate, residual_scale=0.5, next_weight=wn)
        back = cuda_lib.moe_norm_out_backward(dr, y, ry, w, gate=gate, residual_scale=0.5, dn=dn, r=r, rstd_r=rr,
                                              next_weight=wn)
        m, rx = cuda_lib.moe_norm_in(x, w)
        return (r, n, ry, rr, *back, m, rx, *cuda_lib.moe_norm_in_backward(dn, x, rx, w, dresidual=back[0]))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t in (x, y, dr, dn, w, wn, gate):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
