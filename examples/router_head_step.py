"""A learner's steps on the cross entropy of the next tokens, with the router trained and no logits in memory.

    x -> moe_norm_in -> router -> moe_route_topk, moe_balance_loss -> moe_expert_forward
      -> moe_norm_out (residual, final norm) -> head_logprobs
      -> gradients back through the head, the norms, the experts and the router.

The batch is packed sequences with padding: padding tokens have no target, do not count in the balance loss and
take no part in the head's products.  The optimiser and the router's own product are plain torch; run as a script
it prints the losses:

    python examples/router_head_step.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_w4a4_moe_quantize_gb300 as lib  # noqa: E402
from nvfp4_w4a4_moe_quantize_gb300 import synthetic as S  # noqa: E402

IGNORE = -100


class Learner:
    """One block and a head, with the state that a step needs."""

    def __init__(self, shape: S.MoEShape, vocab: int, seed: int = 0):
        x, _, w13, w2 = S.moe_inputs(shape, seed)
        g = torch.Generator().manual_seed(seed + 8_000_001)   # apart from the workload's own seeds
        dev = "cuda"
        self.shape, self.vocab = shape, vocab
        self.x = x.to(dev)
        self.params = {
            "norm_in": torch.ones(shape.H, device=dev),
            "norm_out": torch.full((shape.H,), 0.5, device=dev),
            "norm_final": torch.ones(shape.H, device=dev),
            "w13": w13.to(dev).float(), "w2": w2.to(dev).float(),
            "router": (torch.randn(shape.E, shape.H, generator=g) * 0.05).to(dev),
            "head": (torch.randn(vocab, shape.H, generator=g) * 0.08).to(dev),
        }

    def step(self, targets, sequences, balance: float = 0.01, lr: float = 0.0, seed: int = 0):
        """One step; returns (mean cross entropy, balance losses, tokens of every expert, gradients, what the
        router's and the head's gradients were computed from)."""
        p, s, x = self.params, self.shape, self.x
        valid = targets != IGNORE
        w13, w2 = p["w13"].bfloat16(), p["w2"].bfloat16()
        weights, weights_t = lib.moe_prepare_weights(w13, w2), lib.moe_prepare_weights_backward(w13, w2)
        # forward
        n, rstd_x = lib.moe_norm_in(x, p["norm_in"])
        logits = n.float() @ p["router"].t()
        ids, rw = lib.moe_route_topk(logits, s.k)
        bal, counts, _, tokens = lib.moe_balance_loss(logits, ids, sequences=sequences, valid=valid)
        ws = lib.moe_forward_workspace(x.shape[0], s.k, weights, x.device)
        y = lib.moe_expert_forward(n, ids, rw, weights, workspace=ws)
        r, h, rstd_y, rstd_r = lib.moe_norm_out(x, y, p["norm_out"], next_weight=p["norm_final"])
        head = p["head"].bfloat16()
        logprob, lse, _ = lib.head_logprobs(h, head, targets, ignore_index=IGNORE, entropy=False)
        scored = valid.sum()
        # backward
        dlogprob = -valid.float() / scored
        dh, dhead = lib.head_logprobs_backward(h, head, lse, targets, dlogprob, ignore_index=IGNORE)
        grads = {"head": dhead.float()}
        dx, dy, grads["norm_out"], _, grads["norm_final"] = lib.moe_norm_out_backward(
            None, y, rstd_y, p["norm_out"], dn=dh, r=r, rstd_r=rstd_r, next_weight=p["norm_final"])
        dn, dw, grads["w13"], grads["w2"] = lib.moe_expert_backward(dy, n, rw, weights, weights_t, ws, seed=seed)
        dbal = torch.full_like(bal, balance / bal.shape[0])
        dlogits = lib.moe_router_backward(logits, ids, dw, dloss=dbal, counts=counts, tokens=tokens,
                                          sequences=sequences, valid=valid)
        grads["router"] = dlogits.t() @ n.float()
        dn = (dn.float() + dlogits @ p["router"]).bfloat16()
        dx, grads["norm_in"] = lib.moe_norm_in_backward(dn, x, rstd_x, p["norm_in"], dresidual=dx)
        grads["x"] = dx
        parts = dict(h=h, head=head, n=n, logits=logits, ids=ids, dw=dw, dbal=dbal, valid=valid)
        for k in p:
            p[k] -= lr * grads[k]
        return -logprob.sum() / scored, bal, counts, grads, parts


def batch(shape: S.MoEShape, vocab: int, seed: int = 0):
    """Targets of three packed sequences with padding behind each of them."""
    g = torch.Generator().manual_seed(seed + 8_000_002)
    targets = torch.randint(0, vocab, (shape.T,), generator=g, dtype=torch.int32)
    cuts = [0, shape.T // 4, shape.T // 2, shape.T]
    for end in cuts[1:]:
        targets[end - 7:end] = IGNORE
    return targets.cuda(), torch.tensor(cuts, dtype=torch.int32, device="cuda")


def run(steps: int = 8, vocab: int = 4099, seed: int = 0):
    """Trains on one batch; returns the cross entropies of the steps."""
    shape = S.WORKLOADS["tiny"]
    learner = Learner(shape, vocab, seed)
    targets, sequences = batch(shape, vocab, seed)
    losses = []
    for i in range(steps):
        loss, bal, counts, _, _ = learner.step(targets, sequences, lr=0.5, seed=i)
        losses.append(loss.item())
        print(f"step {i}: cross entropy {loss.item():.4f}, balance {bal.mean().item():.4f}, tokens of the busiest "
              f"expert {int(counts.sum(0).max())}")
    if lib.nvfp4_status_check() != lib.Status.OK:
        raise RuntimeError("a kernel reported an error")
    return losses


if __name__ == "__main__":
    run(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
