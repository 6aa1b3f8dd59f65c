"""A mixture-of-experts block trained with BF16 products of ragged groups.

    python examples/train_moe.py [--tokens 4096] [--steps 20]

    x -> rms_norm -> router logits -> moe_route_topk
      -> rows sorted by expert (no padding) -> m_grouped_bf16_gemm_nt_ragged
      -> swiglu, weighted by the router -> m_grouped_bf16_gemm_nt_ragged
      -> each token's rows added up (moe_combine) -> + x

and back: m_grouped_bf16_gemm_nn_ragged for the rows, k_grouped_bf16_gemm_tn for
the experts' weights, swiglu_bwd (which also gives the gradient of the router's
weights), moe_route_topk_bwd and rms_norm_bwd.  The sort of the rows, the router's
own small products and the optimizer are plain torch.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_gemm_x128_amd as mg  # noqa: E402

BF16 = torch.bfloat16


def _room(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class MoEBlock(torch.autograd.Function):
    """x [T, C] BF16, weights of the norm [C], the router [E, C], the experts' gate and
    up [E, 2 I, C] and down [E, C, I] projections -> x + the experts' weighted sum."""

    @staticmethod
    def forward(ctx, x, w_norm, w_router, w_up, w_down, choices):
        (T, C), (E, two_i, _) = x.shape, w_up.shape
        h = mg.rms_norm(x, w_norm, y=_room(T, C))
        logits = mg.bf16_gemm_nt(h, w_router, None, _room(T, E, dtype=torch.float32))
        idx, weights = _room(T, choices, dtype=torch.int32), _room(T, choices, dtype=torch.float32)
        mg.moe_route_topk(logits, idx, weights, score="sigmoid")
        # rows by expert: order[i] is the (token, choice) pair of row i, slot[t, j] the row of a pair
        expert, order = idx.flatten().sort(stable=True)
        slot = torch.empty_like(order).scatter_(0, order, torch.arange(T * choices, device="cuda")).to(torch.int32)
        slot = slot.view(T, choices)
        offsets = torch.searchsorted(expert, torch.arange(E + 1, dtype=torch.int32, device="cuda")).to(torch.int32)
        token, row_weights = order // choices, weights.flatten()[order]
        rows = h[token]
        up = mg.m_grouped_bf16_gemm_nt_ragged(rows, w_up, _room(T * choices, two_i), offsets)
        act = mg.swiglu(up, y=_room(T * choices, two_i // 2), row_weights=row_weights)
        down = mg.m_grouped_bf16_gemm_nt_ragged(act, w_down, _room(T * choices, C), offsets)
        ones = torch.ones_like(weights)
        y = mg.moe_combine(down[None], slot, ones, _room(T, C))
        ctx.save_for_backward(x, w_norm, w_router, w_up, w_down, h, logits, idx, rows, up, act, offsets, token, slot,
                              row_weights, ones)
        return x + y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        (x, w_norm, w_router, w_up, w_down, h, logits, idx, rows, up, act, offsets, token, slot, row_weights,
         ones) = ctx.saved_tensors
        (T, C), E = x.shape, w_up.shape[0]
        grad = grad.contiguous()
        d_down = grad[token]
        d_act = mg.m_grouped_bf16_gemm_nn_ragged(d_down, w_down, torch.empty_like(act), offsets)
        dw_down = mg.k_grouped_bf16_gemm_tn(d_down, act, torch.empty_like(w_down), offsets)
        d_row_weights = torch.empty_like(row_weights)
        d_up = mg.swiglu_bwd(up, d_act, torch.empty_like(up), row_weights=row_weights, grad_row_weights=d_row_weights)
        dw_up = mg.k_grouped_bf16_gemm_tn(d_up, rows, torch.empty_like(w_up), offsets)
        d_rows = mg.m_grouped_bf16_gemm_nn_ragged(d_up, w_up, torch.empty_like(rows), offsets)
        d_h = mg.moe_combine(d_rows[None], slot, ones, _room(T, C)).float()
        d_logits = mg.moe_route_topk_bwd(logits, idx, d_row_weights[slot.long()], torch.empty_like(logits), score="sigmoid")
        dw_router = torch.matmul(d_logits.t().contiguous(), h.float())
        d_h = d_h + torch.matmul(d_logits, w_router.float())
        dx, dw_norm = torch.empty_like(x), _room(C, dtype=torch.float32)
        workspace = _room(mg.rms_norm_bwd_workspace(T, C) // 4, dtype=torch.float32)
        mg.rms_norm_bwd(d_h, x, w_norm, dx, grad_weight=dw_norm, workspace=workspace, grad_h=grad)
        return dx, dw_norm, dw_router, dw_up, dw_down, None


def block_weights(C, E, I, gen):
    """Random weights (norm F32, the others BF16) that ask for gradients."""
    def normal(*shape):
        return (torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(BF16).requires_grad_()

    return (torch.ones(C, device="cuda").requires_grad_(), normal(E, C), normal(E, 2 * I, C), normal(E, C, I))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--inter", type=int, default=512)
    ap.add_argument("--choices", type=int, default=4)
    args = ap.parse_args()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    weights = block_weights(args.hidden, args.experts, args.inter, gen)
    teacher = [w.detach() for w in block_weights(args.hidden, args.experts, args.inter, gen)]
    optimizer = torch.optim.Adam(weights, lr=2e-3)
    for step in range(args.steps):
        x = torch.randn(args.tokens, args.hidden, generator=gen, device="cuda").to(BF16)
        with torch.no_grad():
            want = MoEBlock.apply(x, *teacher, args.choices)
        loss = (MoEBlock.apply(x, *weights, args.choices).float() - want.float()).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        print(f"step {step}: loss {float(loss.detach()):.4f}", flush=True)


if __name__ == "__main__":
    main()
