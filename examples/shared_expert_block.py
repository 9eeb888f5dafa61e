"""A mixture-of-experts block with a shared expert and norms around it, as a server runs it, and
a dense block trained with its activations kept in 8 bits.

Serving (Block): with r the residual stream and n its normed rows,
    y = experts(n) by gate(n . router^T) + shared(n),
    r' = r + sigmoid(n . w_gate) norm(y),  n' = norm(r') for the next block

Training (train_step): a gated feed-forward block between the same norms, through autograd.

Run with:  python examples/shared_expert_block.py   (needs a GB300 and the built library)
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_moe_grouped_route_gb300 as q  # noqa: E402


class Block:
    """One block's weights: an NVFP4MoE, router [E][H], the shared expert's w13 [2I][H] and w2 [H][I],
    its gate's row w_gate [H], the norm after the block and the one before the next, all bf16."""

    def __init__(self, moe, router, top_k, w13, w2, w_gate, post_weight, next_weight):
        self.moe, self.router, self.top_k = moe, router, top_k
        self.w13, self.w2, self.w_gate = w13, w2, w_gate
        self.post_weight, self.next_weight = post_weight, next_weight

    def __call__(self, r, n):
        """(r, n) [M][H] bf16 of this block -> (r, n) of the next."""
        ids, weights = q.moe_gate(n @ self.router.t(), self.top_k)
        y = self.moe(n, ids, weights) + q.qmoe_gated_ffn(n, self.w13, self.w2)
        out, n, _, _ = q.qmoe_block_norm(y, residual=r, gate=n @ self.w_gate[:, None],
                                         gating=q.QMOE_GATING_SIGMOID, post_weight=self.post_weight,
                                         pre_weight=self.next_weight)
        return out, n


def dense_block(x, w, checkpoint):
    """A dense block of the leaves w: what stands between two values of the residual stream."""
    n = q.qmoe_block_norm(x, pre_weight=w["pre"])[1]
    y = q.qmoe_gated_ffn(n, w["w13"], w["w2"], checkpoint=checkpoint)
    return q.qmoe_block_norm(y, residual=x, gate=w["gate"], post_weight=w["post"])[0]


def train_step(x, want, w, checkpoint=8):
    """(loss, gradients of the leaves w) of the mean squared error."""
    loss = (dense_block(x, w, checkpoint).float() - want).square().mean()
    return loss.detach(), dict(zip(w, torch.autograd.grad(loss, list(w.values()))))


def leaves(H, I, generator=None, device="cuda"):
    def rand(*shape):
        return torch.randn(*shape, generator=generator, device=device)
    w = {"pre": torch.ones(H, device=device), "w13": (rand(2 * I, H) * H ** -0.5).bfloat16(),
         "w2": (rand(H, I) * I ** -0.5).bfloat16(), "post": torch.ones(H, device=device),
         "gate": torch.full((1, H), 0.5, device=device)}
    return {k: v.requires_grad_(True) for k, v in w.items()}


def main():
    from qmoe_inputs import CONFIGS, make_inputs
    torch.manual_seed(0)
    dev, bf16 = "cuda", torch.bfloat16
    li = make_inputs(CONFIGS[0], "cpu").to(dev)
    H, I, E, M = li.cfg.H, 2 * li.cfg.I, li.cfg.E, 6
    block = Block(q.NVFP4MoE(li.w13, li.s13, li.gs13, li.w2, li.s2, li.gs2),
                  torch.randn(E, H, device=dev).to(bf16), li.cfg.top_k,
                  (torch.randn(2 * I, H, device=dev) * H ** -0.5).to(bf16),
                  (torch.randn(H, I, device=dev) * I ** -0.5).to(bf16),
                  (torch.randn(H, device=dev) * H ** -0.5).to(bf16),
                  torch.ones(H, device=dev, dtype=bf16), torch.ones(H, device=dev, dtype=bf16))
    r = torch.randn(M, H, device=dev).to(bf16)
    _, n, _, _ = q.qmoe_block_norm(r, pre_weight=block.next_weight)
    for _ in range(3):
        r, n = block(r, n)
    print("served blocks:", tuple(r.shape), "rms %.3f" % r.float().square().mean().sqrt())

    teacher, w = leaves(128, 256), leaves(128, 256)
    for step in range(20):
        x = torch.randn(256, 128, device=dev).to(bf16)
        with torch.no_grad():
            want = dense_block(x, teacher, 16).float()
        loss, grads = train_step(x, want, w)
        with torch.no_grad():
            for k, v in w.items():
                v -= 0.5 * grads[k].to(v.dtype)
        if step % 5 == 4:
            print("step %2d  loss %.4f" % (step + 1, loss))


if __name__ == "__main__":
    main()
