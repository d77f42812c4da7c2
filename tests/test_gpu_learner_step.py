"""The learner's step of examples/learner_step.py: every operator around the expert block in one
path.  The gradients of the parts that are not quantised are checked against float64
differences of the same step's own forward; a few steps lower the loss."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_steps_lower_the_loss(cuda_lib):
    import learner_step
    losses = learner_step.run(steps=6)
    assert all(l == l and l < float("inf") for l in losses)
    assert losses[-1] < losses[0]


def test_gradient_of_the_final_norm_and_head(cuda_lib):
    """dL/d(norm_final) and dL/d(head) of one step against differences in float64 of the loss as a
    function of them, from the step's own hidden states (BF16 activations and logits are the
    difference: 2^-8 of each term, so 2% of the gradient's norm)."""
    import learner_step
    from nvfp4_w4a4_moe_quantize_gb300 import synthetic as S
    lib, shape, V = cuda_lib, S.WORKLOADS["tiny"], 1031
    learner = learner_step.Learner(shape, V)
    teacher = (2.0 * torch.randn(shape.T, V, generator=torch.Generator().manual_seed(3))).bfloat16().cuda()
    _, _, _, top, ids = lib.token_logprobs(teacher, top_k=16)
    actions = ids[:, 1].contiguous()
    adv = torch.randn(shape.T, generator=torch.Generator().manual_seed(4)).cuda()
    _, _, _, grads = learner.step(ids, top, actions, adv)
    p, x = learner.params, learner.x
    # the same forward up to the final norm, then float64
    w13, w2 = p["w13"].bfloat16(), p["w2"].bfloat16()
    n, _ = lib.moe_norm_in(x, p["norm_in"])
    eid, rw = lib.moe_route_topk(n.float() @ learner.router.t(), shape.k)
    y = lib.moe_expert_forward(n, eid, rw, lib.moe_prepare_weights(w13, w2))
    gate = torch.sigmoid(n.float() @ learner.gate_w)
    r, _, _, _ = lib.moe_norm_out(x, y, p["norm_out"], gate=gate)
    r = r.double()
    nf = p["norm_final"].double().requires_grad_()
    head = p["head"].bfloat16().double().requires_grad_()
    h = r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt() * nf
    lp = torch.log_softmax(h @ head.t(), 1)
    q = top.double().exp()
    at = lp.gather(1, ids.long())
    mask = torch.ones_like(lp).scatter_(1, ids.long(), 0.0)
    pr = (lp.exp() * mask).sum(1)
    qr = (1 - q.sum(1)).clamp(min=0)
    kl = (q * (top.double() - at)).sum(1) + torch.xlogy(qr, qr) - qr * pr.log()
    loss = kl.mean() - (adv.double() * lp.gather(1, actions.long()[:, None]).squeeze(1)).mean()
    want = torch.autograd.grad(loss, (nf, head))
    for name, w in zip(("norm_final", "head"), want):
        err = (grads[name].double() - w).norm() / w.norm()
        assert err < 0.02, (name, err.item())
