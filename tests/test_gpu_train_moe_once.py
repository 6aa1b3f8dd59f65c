"""The training example's block refuses a second derivative, which its backward
pass does not have, and makes its weights' gradients in their own type."""

import os
import sys

import pytest

from helpers import say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_no_second_derivative():
    say("MoE block: a second derivative is refused")
    from train_moe import BF16, MoEBlock, block_weights

    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    weights = block_weights(128, 8, 64, gen)
    x = torch.randn(40, 128, generator=gen, device="cuda").to(BF16).requires_grad_()
    y = MoEBlock.apply(x, *weights, 2).float().square().sum()
    (gx,) = torch.autograd.grad(y, x, create_graph=True)
    with pytest.raises(RuntimeError, match="twice"):
        (gx.float().square().sum() + x.float().pow(3).sum()).backward()


def test_weight_gradients_are_rounded_once(monkeypatch):
    say("MoE block: weight gradients in BF16 from the products themselves")
    import moe_grouped_gemm_x128_amd as mg
    from train_moe import BF16, MoEBlock, block_weights

    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    weights = block_weights(128, 8, 64, gen)
    x = torch.randn(40, 128, generator=gen, device="cuda").to(BF16).requires_grad_()
    made, call = [], mg.k_grouped_bf16_gemm_tn
    monkeypatch.setattr(mg, "k_grouped_bf16_gemm_tn", lambda *a, **kw: (made.append(call(*a, **kw)), made[-1])[1])
    MoEBlock.apply(x, *weights, 2).float().square().sum().backward()
    assert [d.dtype for d in made] == [BF16, BF16]
    assert torch.equal(weights[3].grad, made[0]) and torch.equal(weights[2].grad, made[1])
