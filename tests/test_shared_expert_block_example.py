"""examples/shared_expert_block.py runs, and its gradients are those of its definition."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    path = os.path.join(ROOT, "examples", "shared_expert_block.py")
    spec = importlib.util.spec_from_file_location("shared_expert_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_it_runs(example, capsys):
    example.main()
    said = capsys.readouterr().out
    assert "served blocks" in said and said.count("loss") == 4


@pytest.mark.parametrize("checkpoint", [16, 8])
def test_gradients(example, checkpoint):
    """Against the definition in 64 bits, in the 2-norm: values pass through five to eight bf16
    roundings (about 2^-9.8 each) and, in 8 bits, steps of about 2^-6.5 of a block's root mean
    square, while a missing or doubled term is of the order of 1."""
    g = torch.Generator(device="cuda").manual_seed(3)
    w = example.leaves(128, 264, g)
    x = torch.randn(90, 128, generator=g, device="cuda").bfloat16()
    want = torch.randn(90, 128, generator=g, device="cuda")
    loss, grads = example.train_step(x, want, w, checkpoint)
    v = {k: t.detach().double().requires_grad_(True) for k, t in w.items()}

    def rms(t):
        return t / torch.sqrt(t.square().mean(1, keepdim=True) + 1e-6)
    ug = (rms(x.double()) * v["pre"]) @ v["w13"].t()
    y = (torch.nn.functional.silu(ug[:, 264:]) * ug[:, :264]) @ v["w2"].t()
    out = x.double() + v["gate"] * rms(y) * v["post"]
    ref = (out - want.double()).square().mean()
    ref.backward()
    tol = 2.0 ** -4 if checkpoint == 8 else 2.0 ** -5
    assert abs(float(loss) - float(ref.detach())) <= tol * float(ref.detach())
    for k, t in grads.items():
        assert (t.double() - v[k].grad).norm() <= tol * v[k].grad.norm(), k
