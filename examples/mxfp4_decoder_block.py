"""A decoder block's feed-forward path in MXFP4: a projection trained for a few
steps with every product in 4 bits, then a mixture-of-experts layer that serves
a batch of tokens with the expert weights in 4 bits.

    python examples/mxfp4_decoder_block.py [--tokens 8] [--hidden 1024]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_dg_amd as dg  # noqa: E402


class Projection(torch.autograd.Function):
    """y = x . w^T with x, w and dy quantised along each product's own
    contraction axis; one reading of a tensor gives both of its directions."""

    @staticmethod
    def forward(ctx, x, w):
        qx, sx, qxt, sxt = dg.to_mxfp4_both(x)
        qw, sw, qwt, swt = dg.to_mxfp4_both(w)
        ctx.save_for_backward(qxt, sxt, qwt, swt)
        return dg.mxfp4_gemm_nt(qx, qw, sx, sw)

    @staticmethod
    def backward(ctx, dy):
        qxt, sxt, qwt, swt = ctx.saved_tensors
        qd, sd, qdt, sdt = dg.to_mxfp4_both(dy.contiguous())
        return dg.mxfp4_gemm_nt(qd, qwt, sd, swt), dg.mxfp4_gemm_nt(qdt, qxt, sdt, sxt)


def quantise_experts(w):
    """[E, N, K] -> codes [E, N, K / 2] and scales [E, ceil(K / 128), N]."""
    parts = [dg.to_mxfp4(e) for e in w]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def train(hidden, steps, rows=512):
    """Fit y = x . target^T; returns the losses and the trained weight."""
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    target = rand(hidden, hidden) * hidden ** -0.5
    master = torch.zeros(hidden, hidden, device="cuda")  # FP32 weights, BF16 in the products
    losses = []
    for _ in range(steps):
        x = rand(rows, hidden).to(torch.bfloat16)
        w = master.to(torch.bfloat16).requires_grad_()
        y = Projection.apply(x, w)
        loss = (y.float() - x.float() @ target.t()).square().mean()
        loss.backward()
        master -= 0.25 * hidden * w.grad.float()
        losses.append(loss.item())
    return losses, master.to(torch.bfloat16)


class Block:
    """x + projection, then x + experts, for up to 64 tokens."""

    def __init__(self, projection, hidden, experts, inner, k, tokens):
        g = torch.Generator(device="cuda").manual_seed(1)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
        self.w, self.sw = dg.to_mxfp4(projection)
        self.router = rand(hidden, experts) * hidden ** -0.5
        gate_up = rand(experts, 2 * inner, hidden) * hidden ** -0.5  # row 2i gate, 2i + 1 up
        down = rand(experts, hidden, inner) * inner ** -0.5
        self.w13, self.s13 = quantise_experts(gate_up)
        self.w2, self.s2 = quantise_experts(down)
        self.k = k
        self.workspace = dg.alloc_workspace(max(
            dg.dg_mxfp4_gemm_nt_bf16a_workspace_bytes(tokens, hidden, hidden),
            dg.dg_moe_layer_workspace_bytes(tokens, experts, k, hidden, inner)))

    def __call__(self, x):
        T = x.shape[0]
        p = torch.empty_like(x)
        dg.dg_mxfp4_gemm_nt_bf16a(p, x, self.w, self.sw, workspace=self.workspace)
        x = x + p
        y = torch.empty_like(x)
        ids = torch.empty(T, self.k, dtype=torch.int32, device=x.device)
        weights = torch.empty(T, self.k, device=x.device)
        dg.dg_moe_layer(y, x, self.w13, self.w2, self.s13, self.s2, ids, weights,
                        logits=x.float() @ self.router, workspace=self.workspace)
        return x + y, ids, weights


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=768)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--k", type=int, default=4)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args(argv)
    losses, w = train(a.hidden, a.steps)
    print("projection loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], a.steps))
    block = Block(w, a.hidden, a.experts, a.inner, a.k, a.tokens)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    y, ids, weights = block(x)
    print("token 0: experts %s, weights %s, output norm %.3f" % (
        ids[0].tolist(), ["%.3f" % v for v in weights[0].tolist()], y[0].float().norm().item()))
    return losses, block, x, y, ids, weights


if __name__ == "__main__":
    main()
