"""A mixture-of-experts block from the library's operators, as a server and as a trainer
run it.

Serving (ServedBlock): a projection shared by all requests with a low-rank adapter each,
the router's gate, and the NVFP4 expert layer:
    y = x + proj(x) + adapter(x),  out = y + experts(y) by gate(y . router^T)

Training (forward and backward): experts in bf16, one matrix each, run per expert on the
tokens in expert order, with explicit gradients of the tokens, the router and the experts:
    out[m] = sum_k w[m][k] (x[m] . W[ids[m][k]]^T),  ids, w = gate(x . router^T)

Run with:  python examples/moe_block.py   (needs a GB300 and the built library)
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_moe_grouped_route_gb300 as q  # noqa: E402


class ServedBlock:
    """One block's weights and workspaces.  moe: an NVFP4MoE of the experts; proj [H][H],
    lora_a [L][R][H], lora_b [L][H][R] bf16, scales fp32 [L]; router [E][H] bf16 with a
    selection bias fp32 [E]."""

    def __init__(self, moe, proj, lora_a, lora_b, scales, router, bias, top_k, n_group=1,
                 topk_group=1, scale=1.0):
        self.moe, self.proj, self.router, self.bias = moe, proj, router, bias
        self.lora_a, self.lora_b, self.scales = lora_a, lora_b, scales
        self.top_k, self.n_group, self.topk_group, self.scale = top_k, n_group, topk_group, scale

    def __call__(self, x, adapter_ids):
        """x [M][H] bf16, adapter_ids int32 [M] (-1: none) -> [M][H] bf16."""
        y = q.qmoe_lora_linear(x, self.proj, self.lora_a, self.lora_b, adapter_ids, self.scales,
                               base=x)
        ids, weights = q.moe_gate(y @ self.router.t(), self.top_k, scoring=q.QMOE_GATE_SIGMOID,
                                  bias=self.bias, n_group=self.n_group,
                                  topk_group=self.topk_group, scale=self.scale)
        return y + self.moe(y, ids, weights)


def forward(x, router, experts, top_k):
    """x [M][H] bf16, router [E][H] fp32, experts [E][H][H] bf16 -> (out [M][H], saved)."""
    E = experts.shape[0]
    logits = x.float() @ router.t()
    ids, weights = q.moe_gate(logits, top_k)
    xs, offsets, sorted_pair, pair_pos = q.moe_sort_tokens(x, ids, E)
    ends = offsets.tolist()  # the experts' row ranges, for the products below
    y = torch.zeros_like(xs)
    for e in range(E):
        rows = slice(ends[e], ends[e + 1])
        torch.matmul(xs[rows], experts[e].t(), out=y[rows])
    out = q.moe_unsort_tokens(y, pair_pos, weights)
    return out, (x, router, experts, logits, ids, weights, xs, y, ends, sorted_pair, pair_pos)


def backward(dout, saved):
    """Gradients of x, router and experts from the gradient of out."""
    x, router, experts, logits, ids, weights, xs, y, ends, sorted_pair, pair_pos = saved
    dy, dweights = q.moe_unsort_tokens_backward(dout, y, sorted_pair, pair_pos, weights)
    dxs, dexperts = torch.zeros_like(xs), torch.empty_like(experts)
    for e in range(experts.shape[0]):
        rows = slice(ends[e], ends[e + 1])
        torch.matmul(dy[rows], experts[e], out=dxs[rows])
        torch.matmul(dy[rows].t(), xs[rows], out=dexperts[e])
    dlogits = q.moe_gate_backward(dweights, logits, ids)
    dx = q.moe_sort_tokens_backward(dxs, pair_pos).float() + dlogits @ router
    return dx, dlogits.t() @ x.float(), dexperts


def main():
    from qmoe_inputs import CONFIGS, make_inputs
    torch.manual_seed(0)
    dev, bf16 = "cuda", torch.bfloat16
    li = make_inputs(CONFIGS[0], "cpu").to(dev)
    c = li.cfg
    L, R, M = 4, 16, 6
    block = ServedBlock(
        q.NVFP4MoE(li.w13, li.s13, li.gs13, li.w2, li.s2, li.gs2),
        (torch.randn(c.H, c.H, device=dev) * c.H ** -0.5).to(bf16),
        (torch.randn(L, R, c.H, device=dev) * c.H ** -0.5).to(bf16),
        (torch.randn(L, c.H, R, device=dev) * R ** -0.5).to(bf16), torch.full((L,), 0.5, device=dev),
        torch.randn(c.E, c.H, device=dev).to(bf16), torch.zeros(c.E, device=dev), c.top_k, 2, 1)
    x = torch.randn(M, c.H, device=dev).to(bf16)
    out = block(x, torch.tensor([0, 3, -1, 1, 1, 2], dtype=torch.int32, device=dev))
    print("served block:", tuple(out.shape), "rms %.3f" % out.float().square().mean().sqrt())

    E, H, M, top_k = 8, 64, 256, 2
    teacher = (torch.randn(E, H, H, device=dev) * H ** -0.5).to(bf16)
    experts = (teacher.float() + 0.3 * H ** -0.5 * torch.randn(E, H, H, device=dev)).to(bf16)
    router = torch.randn(E, H, device=dev) * H ** -0.5
    for step in range(20):
        x = torch.randn(M, H, device=dev).to(bf16)
        want, _ = forward(x, router, teacher, top_k)
        out, saved = forward(x, router, experts, top_k)
        diff = out.float() - want.float()
        _, drouter, dexperts = backward((2 * diff / M).to(bf16), saved)
        experts = (experts.float() - 0.5 * dexperts.float()).to(bf16)
        router = router - 0.01 * drouter
        if step % 5 == 4:
            print("training step %2d: loss %.5f" % (step + 1, diff.square().sum(1).mean()))


if __name__ == "__main__":
    main()
