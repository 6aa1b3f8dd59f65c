"""The block of examples/train_moe.py: its output and gradients against the same
block in float64 with torch's autograd, the routing choice as the block made it.

Each rounding to BF16 is off by at most 2^-8 of a value, an rms of 2^-8 / sqrt(3); a
path through the block and back holds at most 12 of them (norm, rows, both
products, activation, sum and output; the same back): the normalised difference is
at most half the sum of their squares, 3.1e-5, doubled for the products between
them.  The router's gradient is what is left of that of the weights when their mean
goes off: at least half in the mean square, so twice the bound again, and twice for
the weight as one factor of every product.  The output and the gradient of x are
what the block adds to a stream, rounded with it: beside the parts' bound that one
rounding counts, 2^-8 / sqrt(3) of the whole."""

import os
import sys

import pytest

from helpers import norm_diff, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

DIFF = 6.2e-5


def _plain(x, w_norm, w_router, w_up, w_down, idx):
    h = x / (x.square().mean(dim=-1, keepdim=True) + 1e-6).sqrt() * w_norm
    s = torch.sigmoid(h @ w_router.t()).gather(1, idx)
    wgt = s / s.sum(dim=1, keepdim=True)
    I = w_down.shape[2]
    y = x
    for e in range(w_up.shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        u = h[t] @ w_up[e].t()
        act = torch.nn.functional.silu(u[:, :I]) * u[:, I:] * wgt[t, j][:, None]
        y = y.index_add(0, t, act @ w_down[e].t())
    return y


@pytest.mark.parametrize("T,C,E,I,k", [(300, 256, 8, 128, 2), (37, 128, 16, 192, 4), (1, 128, 4, 64, 2)])
def test_gradients_match_float64(T, C, E, I, k, monkeypatch):
    say(f"MoE block T={T} C={C} E={E} I={I} k={k}")
    import moe_grouped_gemm_x128_amd as mg
    from train_moe import BF16, MoEBlock, block_weights

    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    weights = block_weights(C, E, I, gen)
    x = (torch.randn(T, C, generator=gen, device="cuda") * 2).to(BF16).requires_grad_()
    grad = torch.randn(T, C, generator=gen, device="cuda").to(BF16)
    seen = []
    route = mg.moe_route_topk
    monkeypatch.setattr(mg, "moe_route_topk", lambda lg, idx, *a, **kw: (seen.append(idx), route(lg, idx, *a, **kw))[1])
    got = MoEBlock.apply(x, *weights, k)
    got.backward(grad)
    ref = [t.detach().double().requires_grad_() for t in (x, *weights)]
    want = _plain(*ref, seen[0].long())
    want.backward(grad.double())
    for name, a, b, past in [("output", got, want, x)] + [
            (n, t.grad, r.grad, grad if n == "x" else None)
            for n, t, r in zip(("x", "norm", "router", "up", "down"), (x, *weights), ref)]:
        a, b, tol = a.detach().double(), b.detach(), DIFF * (4 if name == "router" else 1)
        if past is not None:
            part = b - past.detach().double()
            tol += 0.5 * 2.0 ** -16 / 3 * float(b.square().mean() / part.square().mean())
            a, b = a - past.detach().double(), part
        d = norm_diff(a.cpu().numpy(), b.cpu().numpy())
        say(f"  {name}: normalised difference {d:.2e} of {tol:.1e}")
        assert torch.isfinite(a).all() and d <= tol, name


def test_example_runs():
    say("MoE training example")
    import train_moe

    argv, sys.argv = sys.argv, ["train_moe.py", "--tokens", "200", "--steps", "2", "--hidden", "256", "--experts", "8",
                                "--inter", "128", "--choices", "2"]
    try:
        train_moe.main()
    finally:
        sys.argv = argv


def test_two_backward_passes_give_the_same_bits():
    say("MoE block: the same gradients twice")
    from train_moe import BF16, MoEBlock, block_weights

    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    weights = block_weights(256, 16, 128, gen)
    x = torch.randn(500, 256, generator=gen, device="cuda").to(BF16).requires_grad_()
    grads = []
    for _ in range(2):
        for t in (x, *weights):
            t.grad = None
        MoEBlock.apply(x, *weights, 4).float().square().sum().backward()
        grads.append([t.grad.clone() for t in (x, *weights)])
    assert all(torch.equal(a, b) for a, b in zip(*grads))
