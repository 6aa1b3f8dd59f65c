"""The layer of examples/decode_layer.py against the same layer in float64.

Both use the FP8 weights' values and the layer's own routing choice.  What
remains is the rounding of activations and cache to E4M3 (five casts, each an
rms error of at most 2^-4 / sqrt(3) of a value, 0.036) and to BF16: the
normalised difference of the layer's contribution stays within half the sum of
their squares, 3.3e-3, doubled for the products between them."""

import os
import sys

import numpy as np
import pytest

from helpers import norm_diff, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

DIFF = 6.6e-3


def _weight(w):
    q, sf = w
    big = sf.double().repeat_interleave(128, -2).repeat_interleave(128, -1)[..., :q.shape[-2], :q.shape[-1]]
    return q.view(torch.float8_e4m3fn).double() * big


def _norm(x):
    return x / (x.square().mean(dim=-1, keepdim=True) + 1e-6).sqrt()


def _rotate(x, pos, cos_sin):
    half = x.shape[-1] // 2
    c, s = (t[:, None] for t in cos_sin.double()[pos].split(half, dim=1))
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], dim=-1)


class Plain:
    def __init__(self, layer):
        self.l = layer
        self.w = {n: _weight(getattr(layer, n)) for n in ("w_qkv", "w_out", "w_up", "w_down")}
        self.kv = [(None, None)] * layer.batch
        self.pos = 0

    def forward(self, x, idx):
        l = self.l
        S, n, C = x.shape
        H, G, D = l.heads, l.kv_heads, l.head_dim
        x = x.double().view(S * n, C)
        qkv = (_norm(x) @ self.w["w_qkv"].t()).view(S, n, H + 2 * G, D)
        pos = torch.arange(self.pos, self.pos + n, device="cuda")
        outs = []
        for s in range(S):
            q, k = _rotate(qkv[s, :, :H], pos, l.cos_sin), _rotate(qkv[s, :, H:H + G], pos, l.cos_sin)
            v = qkv[s, :, H + G:]
            ok, ov = self.kv[s]
            k = k if ok is None else torch.cat([ok, k])
            v = v if ov is None else torch.cat([ov, v])
            self.kv[s] = (k, v)
            kk, vv = (t.repeat_interleave(H // G, dim=1).transpose(0, 1).contiguous() for t in (k, v))
            score = torch.matmul(q.transpose(0, 1), kk.transpose(1, 2).contiguous()) * D ** -0.5
            mask = torch.arange(k.shape[0], device="cuda")[None] > pos[:, None]
            score = score.masked_fill(mask[None], -np.inf)
            outs.append(torch.matmul(torch.softmax(score, dim=-1), vv).transpose(0, 1).reshape(n, H * D))
        self.pos += n
        x = x + torch.cat(outs) @ self.w["w_out"].t()
        h = _norm(x)
        s = torch.sigmoid(h @ l.w_router.double().t())
        y = torch.zeros_like(x)
        for j in range(idx.shape[1]):
            e = idx[:, j].long()
            wgt = s.gather(1, e[:, None]) / s.gather(1, idx.long()).sum(dim=1, keepdim=True)
            for g in e.unique().tolist():
                r = torch.nonzero(e == g)[:, 0]
                u = h[r] @ self.w["w_up"][g].t()
                act = torch.nn.functional.silu(u[:, :l.inter]) * u[:, l.inter:]
                y[r] += wgt[r] * (act @ self.w["w_down"][g].t())
        return (x + y).view(S, n, C)


def test_layer_matches_float64():
    say("decode layer: a prompt of 37 tokens, then five single steps")
    from decode_layer import DecodeLayer

    layer = DecodeLayer(batch=3, max_tokens=50, hidden=512, heads=8, kv_heads=2, head_dim=64, experts=16, choices=3,
                        inter=256, page=16, seed=3)
    plain = Plain(layer)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    for n in (37, 1, 1, 1, 1, 1):
        x = torch.randn(3, n, 512, generator=gen, device="cuda").to(torch.bfloat16)
        got = layer.forward(x)
        idx, weights = layer.routes
        assert torch.all(idx >= 0) and torch.allclose(weights.sum(dim=1), torch.ones(3 * n, device="cuda"), atol=1e-6)
        assert all(len(set(r)) == 3 for r in idx.tolist())
        want = plain.forward(x, idx)
        d = norm_diff((got.double() - x.double()).cpu().numpy(), (want - x.double()).cpu().numpy())
        say(f"  n={n}: normalised difference of the layer's contribution {d:.2e}")
        assert torch.all(torch.isfinite(got)) and d <= DIFF
    assert layer.lens.tolist() == [42] * 3


def test_example_runs():
    say("decode layer example")
    import decode_layer

    argv, sys.argv = sys.argv, ["decode_layer.py", "--batch", "4", "--prompt", "20", "--steps", "3"]
    try:
        decode_layer.main()
    finally:
        sys.argv = argv


def test_graph_replays_equal_eager_steps():
    say("decode layer under graph capture")
    from decode_layer import DecodeLayer

    kw = dict(batch=4, max_tokens=64, hidden=512, heads=8, kv_heads=2, head_dim=64, experts=16, choices=3, inter=256,
              page=16, seed=5)
    eager, graphed = DecodeLayer(**kw), DecodeLayer(**kw)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    x = torch.randn(4, 1, 512, generator=gen, device="cuda").to(torch.bfloat16)
    graphed.forward(x)
    eager.forward(x)
    token = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = graphed.forward(token)
    for _ in range(4):
        x = torch.randn(4, 1, 512, generator=gen, device="cuda").to(torch.bfloat16)
        token.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager.forward(x))
        torch.cuda.synchronize()
