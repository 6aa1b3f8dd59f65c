"""One mixture-of-experts transformer layer served from a paged FP8 cache.

    python examples/decode_layer.py [--batch 64] [--prompt 128] [--steps 32]

Every matrix product, cast, cache and routing step is a call of this library:

    x -> norm -> q, k, v projection (per-token cast + FP8 GEMM)
      -> kv_append_fp8: keys rotated into the paged cache, queries rotated
      -> paged_attention_fp8 over the cache -> output projection
      -> norm -> router logits (BF16 GEMM, FP32 out) -> moe_route_topk
      -> moe_dispatch_masked_fp8 -> gate / up GEMM of every expert
      -> silu(gate) * up -> per-token cast -> down GEMM -> moe_combine

The norms, the activation and the residual additions are plain torch.  Weights
are random; the prompt goes through the same calls as a decode step, with as
many queries a sequence as it has tokens.  The decode step is captured into a
hipGraph once and replayed.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_gemm_x128_amd as mg  # noqa: E402


def _quantized(shape, gen, gain=1.0):
    """A random weight [.., N, K] of variance gain / K, as FP8 codes and block scales."""
    w = torch.randn(shape, generator=gen, device="cuda") * (gain / shape[-1] ** 0.5)
    q = torch.empty(shape, dtype=torch.uint8, device="cuda")
    blocks = (-(-shape[-2] // 128), -(-shape[-1] // 128))
    sf = torch.empty(shape[:-2] + blocks, device="cuda")
    mg.per_block_cast_to_fp8(w, q, sf)
    return q, sf


def _norm(x):
    return x * torch.rsqrt(x.float().square().mean(dim=-1, keepdim=True) + 1e-6).to(x.dtype)


class DecodeLayer:
    """Weights, the paged cache of `batch` sequences of up to max_tokens, and the layer's forward."""

    def __init__(self, batch, max_tokens, hidden=1024, heads=16, kv_heads=2, head_dim=128, experts=32, choices=4,
                 inter=512, page=64, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.batch, self.hidden, self.heads, self.kv_heads, self.head_dim = batch, hidden, heads, kv_heads, head_dim
        self.experts, self.choices, self.inter = experts, choices, inter
        self.w_qkv = _quantized(((heads + 2 * kv_heads) * head_dim, hidden), gen)
        self.w_out = _quantized((hidden, heads * head_dim), gen)
        self.w_router = (torch.randn(experts, hidden, generator=gen, device="cuda") / hidden ** 0.5).to(torch.bfloat16)
        self.router_bias = torch.randn(experts, generator=gen, device="cuda") * 0.02
        self.w_up = _quantized((experts, 2 * inter, hidden), gen)
        self.w_down = _quantized((experts, hidden, inter), gen)
        per_seq = -(-max_tokens // page)
        pages = batch * per_seq
        pool = torch.zeros(pages, 2, kv_heads, page, head_dim, dtype=torch.uint8, device="cuda")
        scales = torch.ones(pages, 2, kv_heads, device="cuda")
        self.cache = (pool[:, 0], pool[:, 1], scales[:, 0], scales[:, 1])
        self.table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(batch, per_seq)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.max_tokens = per_seq * page
        freq = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim)
        ang = torch.arange(self.max_tokens, device="cuda", dtype=torch.float64)[:, None] * freq
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        self.routes = None  # the last step's (topk_idx, topk_weights)

    def _linear(self, x, weight):
        """x [M, K] BF16 times an FP8 weight [N, K], BF16 out."""
        (M, K), (w, sfw) = x.shape, weight
        a = torch.empty(M, K, dtype=torch.uint8, device="cuda")
        sfa = torch.empty(K // 128, M, device="cuda").t()
        d = torch.empty(M, w.shape[0], dtype=torch.bfloat16, device="cuda")
        mg.per_token_cast_to_fp8(x, a, sfa)
        return mg.fp8_gemm_nt(a, w, sfa, sfw, None, d)

    def attention(self, x, n):
        """x [batch * n, hidden]: n new tokens of every sequence."""
        S, H, G, D = self.batch, self.heads, self.kv_heads, self.head_dim
        qkv = self._linear(x, self.w_qkv).view(S * n, H + 2 * G, D)
        q = torch.empty(S * n, H, D, dtype=torch.bfloat16, device="cuda")
        cu = torch.arange(0, S * n + 1, n, dtype=torch.int32, device="cuda")
        mg.kv_append_fp8(qkv[:, H:H + G], qkv[:, H + G:], *self.cache, self.table, cu, self.lens, cos_sin=self.cos_sin,
                         q=qkv[:, :H], q_out=q)
        self.lens += n
        out = torch.empty(S, n, H, D, dtype=torch.bfloat16, device="cuda")
        need = mg.paged_attention_fp8_workspace(S, n, H, G, D, self.max_tokens)
        mg.paged_attention_fp8(q.view(S, n, H, D), *self.cache, self.table, self.lens, out, D ** -0.5,
                               workspace=torch.empty(-(-need // 4), device="cuda"))
        return self._linear(out.view(S * n, H * D), self.w_out)

    def moe(self, x):
        T, E, k, I = x.shape[0], self.experts, self.choices, self.inter
        logits = torch.empty(T, E, device="cuda")
        mg.bf16_gemm_nt(x, self.w_router, None, logits)
        idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
        weights = torch.empty(T, k, device="cuda")
        mg.moe_route_topk(logits, idx, weights, bias=self.router_bias, score="sigmoid", n_group=4, topk_group=2,
                          group_top=2)
        self.routes = (idx, weights)
        a = torch.empty(E, T, self.hidden, dtype=torch.uint8, device="cuda")  # every expert could get every token
        sfa = torch.empty(E, T, self.hidden // 128, device="cuda")
        rows = torch.empty(E, dtype=torch.int32, device="cuda")
        slot = torch.empty(T, k, dtype=torch.int32, device="cuda")
        src = torch.empty(E, T, dtype=torch.int32, device="cuda")
        mg.moe_dispatch_masked_fp8(x, idx, a, sfa, rows, slot, src)
        up = torch.empty(E, T, 2 * I, dtype=torch.bfloat16, device="cuda")
        mg.m_grouped_fp8_gemm_nt_masked(a, self.w_up[0], sfa, self.w_up[1], up, rows, T)
        act = torch.nn.functional.silu(up[..., :I]) * up[..., I:]
        b = torch.empty(E, T, I, dtype=torch.uint8, device="cuda")
        sfb = torch.empty(E, T, I // 128, device="cuda")
        mg.per_token_cast_to_fp8(act, b, sfb)
        down = torch.empty(E, T, self.hidden, dtype=torch.bfloat16, device="cuda")
        mg.m_grouped_fp8_gemm_nt_masked(b, self.w_down[0], sfb, self.w_down[1], down, rows, T)
        return mg.moe_combine(down, slot, weights, torch.empty_like(x))

    def forward(self, x):
        """x BF16 [batch, n, hidden]: n new tokens of every sequence -> the layer's output for them."""
        S, n, C = x.shape
        x = x.reshape(S * n, C)
        x = x + self.attention(_norm(x), n)
        x = x + self.moe(_norm(x))
        return x.view(S, n, C)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=128)
    ap.add_argument("--steps", type=int, default=32)
    args = ap.parse_args()
    layer = DecodeLayer(args.batch, args.prompt + args.steps + 4)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(args.batch, args.prompt, layer.hidden, generator=gen, device="cuda").to(torch.bfloat16)
    token = layer.forward(x)[:, -1:].contiguous()
    token = layer.forward(token)  # (once before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(token)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(args.steps):
        graph.replay()
        token.copy_(out)
    torch.cuda.synchronize()
    us = (time.perf_counter() - begin) / args.steps * 1e6
    counts = torch.bincount(layer.routes[0].flatten().long(), minlength=layer.experts)
    print(f"{args.batch} sequences, {int(layer.lens[0])} tokens each: {us:.0f} us a step of one layer, "
          f"{args.batch / us * 1e6:.0f} tokens/s; busiest expert {int(counts.max())} tokens, "
          f"output rms {float(out.float().square().mean().sqrt()):.3f}")


if __name__ == "__main__":
    main()
