"""A learner's steps around the NVFP4 W4A4 expert block: distillation from a teacher's top
tokens with a policy-gradient term.

    x -> moe_norm_in -> route -> moe_expert_forward -> moe_norm_out (gate, residual, final norm)
      -> head -> token_logprobs (policy) and distill_topk_backward (teacher)
      -> gradients back through the head, the norms and the experts.

The teacher's list of every token comes from token_logprobs on the teacher's logits.  The head,
the router and the optimiser are plain torch; run as a script it prints the losses:

    python examples/learner_step.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_w4a4_moe_quantize_gb300 as lib  # noqa: E402
from nvfp4_w4a4_moe_quantize_gb300 import synthetic as S  # noqa: E402


class Learner:
    """One block and a head, with the state that a step needs."""

    def __init__(self, shape: S.MoEShape, vocab: int, seed: int = 0):
        x, _, w13, w2 = S.moe_inputs(shape, seed)
        g = torch.Generator().manual_seed(seed + 7_000_001)   # apart from the workload's own seeds
        dev = "cuda"
        self.shape, self.vocab = shape, vocab
        self.x = x.to(dev)
        self.router = (torch.randn(shape.E, shape.H, generator=g) * 0.05).to(dev)
        self.gate_w = (torch.randn(shape.H, generator=g) * 0.05).to(dev)
        self.params = {
            "norm_in": torch.ones(shape.H, device=dev),
            "norm_out": torch.full((shape.H,), 0.5, device=dev),
            "norm_final": torch.ones(shape.H, device=dev),
            "w13": w13.to(dev).float(), "w2": w2.to(dev).float(),
            "head": (torch.randn(vocab, shape.H, generator=g) * 0.08).to(dev),
        }

    def step(self, teacher_ids, teacher_logprobs, actions, advantages, lr: float = 0.0, seed: int = 0):
        """One step; returns (distillation loss, mean log probability of the actions, entropy, gradients)."""
        p, s, x = self.params, self.shape, self.x
        T = x.shape[0]
        w13, w2 = p["w13"].bfloat16(), p["w2"].bfloat16()
        weights, weights_t = lib.moe_prepare_weights(w13, w2), lib.moe_prepare_weights_backward(w13, w2)
        # forward
        n, rstd_x = lib.moe_norm_in(x, p["norm_in"])
        ids, rw = lib.moe_route_topk(n.float() @ self.router.t(), s.k)
        ws = lib.moe_forward_workspace(T, s.k, weights, x.device)
        y = lib.moe_expert_forward(n, ids, rw, weights, workspace=ws)
        gate = torch.sigmoid(n.float() @ self.gate_w)
        r, h, rstd_y, rstd_r = lib.moe_norm_out(x, y, p["norm_out"], gate=gate, next_weight=p["norm_final"])
        head = p["head"].bfloat16()
        logits = h @ head.t()
        # the policy's terms and the distillation's loss with its gradient
        logprob, lse, entropy, _, _ = lib.token_logprobs(logits, actions)
        dlogits = lib.token_logprobs_backward(logits, lse, actions, -advantages / T)
        loss, dkl = lib.distill_topk_backward(logits, teacher_ids, teacher_logprobs,
                                              torch.full((T,), 1.0 / T, device=x.device), out=logits)
        dlogits = dlogits.float() + dkl.float()
        # backward
        grads = {"head": dlogits.t() @ h.float()}
        dh = (dlogits @ head.float()).bfloat16()
        dx, dy, grads["norm_out"], _, grads["norm_final"] = lib.moe_norm_out_backward(
            None, y, rstd_y, p["norm_out"], gate=gate, dn=dh, r=r, rstd_r=rstd_r, next_weight=p["norm_final"])
        dn, _, grads["w13"], grads["w2"] = lib.moe_expert_backward(dy, n, rw, weights, weights_t, ws, seed=seed)
        dx, grads["norm_in"] = lib.moe_norm_in_backward(dn, x, rstd_x, p["norm_in"], dresidual=dx)
        grads["x"] = dx
        for k in p:
            p[k] -= lr * grads[k]
        return loss.mean(), logprob.mean(), entropy.mean(), grads


def run(steps: int = 8, vocab: int = 4099, seed: int = 0):
    """Distils a random teacher into the block; returns the losses of the steps."""
    shape = S.WORKLOADS["tiny"]
    learner = Learner(shape, vocab, seed)
    g = torch.Generator().manual_seed(seed + 7_000_002)
    teacher = (torch.randn(shape.T, 1, generator=g) + 2.0 * torch.randn(shape.T, vocab, generator=g)).bfloat16().cuda()
    _, _, _, top_logprobs, top_ids = lib.token_logprobs(teacher, top_k=32, entropy=False)
    actions = top_ids[:, 0].contiguous()
    advantages = torch.full((shape.T,), 0.1, device="cuda")
    losses = []
    for i in range(steps):
        loss, logprob, entropy, _ = learner.step(top_ids, top_logprobs, actions, advantages, lr=0.5, seed=i)
        losses.append(loss.item())
        print(f"step {i}: distillation loss {loss.item():.4f}, action log probability {logprob.item():.4f}, "
              f"entropy {entropy.item():.4f}")
    if lib.nvfp4_status_check() != lib.Status.OK:
        raise RuntimeError("a kernel reported an error")
    return losses


if __name__ == "__main__":
    run(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
