"""The training example's block refuses a second derivative, which its backward
pass does not have."""

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
