"""The example block: its serving path against the same block from torch operations and the
layer, its gradients against autograd in 64 bits."""

import importlib.util
import os

import pytest
import torch

import quantized_moe_grouped_route_gb300 as q

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("moe_block",
                                                  os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@gpu
def test_training_gradients():
    m = _example()
    g = torch.Generator(device="cuda").manual_seed(1)
    M, E, H, k = 96, 8, 64, 2
    x = torch.randn(M, H, generator=g, device="cuda").bfloat16()
    router = torch.randn(E, H, generator=g, device="cuda") * H ** -0.5
    experts = (torch.randn(E, H, H, generator=g, device="cuda") * H ** -0.5).bfloat16()
    dout = torch.randn(M, H, generator=g, device="cuda").bfloat16()
    out, saved = m.forward(x, router, experts, k)
    dx, drouter, dexperts = m.backward(dout, saved)
    ids = saved[4].long()

    x64, r64, w64 = (t.double().requires_grad_(True) for t in (x, router, experts))
    logits = x64 @ r64.t()
    w = torch.softmax(torch.gather(logits, 1, ids), 1)
    ref = (w[..., None] * torch.einsum("mh,mkoh->mko", x64, w64[ids])).sum(1)
    (ref * dout.double()).sum().backward()
    # bf16 stands between the stages (y, dy, dxs, the outputs): a handful of roundings of
    # 2^-8 relative to the terms' size, which the root of the sums' squares bounds
    for got, want in ((out, ref), (dx, x64.grad), (drouter, r64.grad), (dexperts, w64.grad)):
        err = (got.double() - want.detach()).norm() / want.detach().norm()
        assert err < 4 * 2.0 ** -8, float(err)


@gpu
def test_served_block():
    from qmoe_inputs import CONFIGS, make_inputs
    m = _example()
    g = torch.Generator(device="cuda").manual_seed(2)
    li = make_inputs(CONFIGS[0], "cpu").to("cuda")
    c, L, R, M = li.cfg, 3, 16, 9

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    moe = q.NVFP4MoE(li.w13, li.s13, li.gs13, li.w2, li.s2, li.gs2)
    proj, a, b = rand(c.H, c.H, std=c.H ** -0.5), rand(L, R, c.H, std=c.H ** -0.5), rand(L, c.H, R)
    scales = torch.full((L,), 0.25, device="cuda")
    router = rand(c.E, c.H)
    block = m.ServedBlock(moe, proj, a, b, scales, router, torch.zeros(c.E, device="cuda"), c.top_k)
    x = rand(M, c.H)
    ad = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    out = block(x, ad)
    x64 = x.double()
    at = ad.clamp(min=0).long()
    t = 0.25 * torch.einsum("mh,mrh->mr", x64, a.double()[at])
    delta = torch.where((ad >= 0)[:, None], torch.einsum("mr,mnr->mn", t, b.double()[at]), 0.0)
    y = q.qmoe_lora_linear(x, proj, a, b, ad, scales, base=x)
    exact = x64 + x64 @ proj.double().t() + delta
    assert (y.double() - exact).norm() / exact.norm() < 2.0 ** -8  # one rounding
    # the choice of experts is not continuous in y, so it is made from this y: the scores with
    # the definition's fp32 operations, ties to the lowest expert
    s = 1.0 / (1.0 + torch.exp(-(y @ router.t()).float()))
    top = torch.sort(s, dim=1, descending=True, stable=True)
    scores, ids = top.values[:, :c.top_k], top.indices[:, :c.top_k].to(torch.int32).contiguous()
    ref = y + moe(y, ids, scores / scores.sum(1, keepdim=True))
    # the routing weights differ in their last bits, the outputs by roundings of them
    err = (out.double() - ref.double()).norm() / ref.double().norm()
    assert err < 2.0 ** -7, float(err)


@gpu
def test_example_runs(capsys):
    _example().main()
    lines = capsys.readouterr().out.splitlines()
    losses = [float(s.split()[-1]) for s in lines if s.startswith("training")]
    assert len(losses) == 4 and losses[-1] < 0.8 * losses[0], lines
