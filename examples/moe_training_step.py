"""A mixture-of-experts layer around the grouped FP8 products: routing, the
layout, activations quantised into it, the experts, and the weighted sum back;
then its gradients, with the gate/up values kept in 8 bits in between.

    python examples/moe_training_step.py [--tokens 1000] [--hidden 1024]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_dg_amd as dg  # noqa: E402


def quantise_experts(w):
    """w [E, N, K] float32 -> codes [E, N, K] and 128 x 128 scales [E, K/128, N/128],
    and those of the transposed weights, which the backward products take."""
    E, N, K = w.shape
    parts = [dg.to_fp8(e.contiguous(), 128) for e in w]
    q, s = (torch.stack([p[i] for p in parts]) for i in range(2))
    qt = torch.empty((E, K, N), dtype=torch.uint8, device=w.device)
    for e in range(E):
        dg.dg_transpose_fp8(qt[e], q[e])
    return q, s, qt, s.transpose(1, 2).contiguous()


def grouped(a, sa, w, sw, m_indices):
    """The rows of a times their experts' weights [E, N, K] -> bfloat16 [M, N]."""
    c = torch.empty((a.shape[0], w.shape[1]), dtype=torch.bfloat16, device=a.device)
    dg.dg_fp8_grouped_gemm_contig(c, a, w, sa, sw, 1, m_indices)
    return c


def weight_gradient(d, sd, x, sx, plan):
    """Per expert d^T . x over its rows (codes [M, N] and [M, K]) -> bfloat16 [E, N, K]."""
    dt, sdt = dg.transpose_fp8_blocks(d, sd, 1, plan.m_indices)
    xt, sxt = dg.transpose_fp8_blocks(x, sx, 128, plan.m_indices)
    out = torch.empty((plan.counts.numel(), d.shape[1], x.shape[1]), dtype=torch.bfloat16,
                      device=d.device)
    dg.dg_fp8_grouped_gemm_k(out, dt, xt, sdt, sxt, 1, plan.offsets)
    return out


class Experts:
    """w13 [E, 2I, H] (row 2i gate, 2i+1 up) and w2 [E, H, I], float32."""

    def __init__(self, w13, w2, k, **routing):
        self.k, self.routing = k, routing
        self.w13, self.w2 = quantise_experts(w13), quantise_experts(w2)

    def forward(self, x, logits, bias=None):
        """x [T, H] bfloat16, logits [T, E] -> y [T, H], and what the backward needs."""
        s = dict(logits=logits)
        s["ids"], s["weights"] = dg.moe_route(logits, self.k, bias=bias, **self.routing)
        s["plan"] = plan = dg.moe_plan(s["ids"], logits.shape[1])
        s["a"], s["sa"] = dg.moe_dispatch_fp8(x, plan)
        gu = grouped(s["a"], s["sa"], *self.w13[:2], plan.m_indices)
        s["h"], s["sh"], s["kept"], s["skept"] = dg.swiglu_fp8(gu, plan.m_indices, keep=True)
        s["c"] = grouped(s["h"], s["sh"], *self.w2[:2], plan.m_indices)
        return dg.moe_combine(s["c"], plan, s["weights"]), s

    def backward(self, dy, s):
        """dy [T, H] bfloat16 -> gradients of x, logits, w13 and w2, and what lies
        between them."""
        plan, (T, H) = s["plan"], dy.shape
        g = {}
        g["dc"], g["sdc"] = torch.empty_like(s["a"]), torch.empty_like(s["sa"])
        g["dweights"] = torch.empty_like(s["weights"])
        dg.dg_moe_combine_backward(g["dc"], g["sdc"], g["dweights"], dy, s["c"], plan.rows, plan.pairs,
                                   s["weights"])
        g["logits"] = torch.empty_like(s["logits"])
        routing = {n: v for n, v in self.routing.items() if n in ("scoring", "renormalise", "scale")}
        dg.dg_moe_route_backward(g["logits"], g["dweights"], s["ids"], s["logits"], **routing)
        g["dh"] = grouped(g["dc"], g["sdc"], *self.w2[2:], plan.m_indices)
        g["dgu"], g["sdgu"] = torch.empty_like(s["kept"]), torch.empty_like(s["skept"])
        g["h"], g["sh"] = torch.empty_like(s["h"]), torch.empty_like(s["sh"])
        dg.dg_swiglu_fp8_backward(g["dgu"], g["sdgu"], g["dh"], s["kept"], s["skept"], g["h"], g["sh"],
                                  plan.m_indices)
        g["rows"] = grouped(g["dgu"], g["sdgu"], *self.w13[2:], plan.m_indices)
        g["x"] = dg.moe_combine(g["rows"], plan)
        g["w2"] = weight_gradient(g["dc"], g["sdc"], g["h"], g["sh"], plan)
        g["w13"] = weight_gradient(g["dgu"], g["sdgu"], s["a"], s["sa"], plan)
        return g


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=1000)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--inner", type=int, default=512)
    p.add_argument("--experts", type=int, default=16)
    p.add_argument("--k", type=int, default=4)
    a = p.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)
    T, H, I, E = a.tokens, a.hidden, a.inner, a.experts
    layer = Experts(rand(E, 2 * I, H) * H ** -0.5, rand(E, H, I) * I ** -0.5, a.k, scoring="sigmoid",
                    scale=2.0)
    x, router, bias = rand(T, H).to(torch.bfloat16), rand(E, H) * H ** -0.5, rand(E) * 0.05
    logits = x.float() @ router.t()
    y, saved = layer.forward(x, logits, bias)
    dy = (rand(T, H) * 1e-3).to(torch.bfloat16)
    grads = layer.backward(dy, saved)
    load = saved["plan"].counts
    print("%d tokens to %d of %d experts, load %d to %d, |y| %.3g, |dx| %.3g, |dw13| %.3g, |dw2| %.3g"
          % (T, a.k, E, load.min(), load.max(), y.float().norm(), grads["x"].float().norm(),
             grads["w13"].float().norm(), grads["w2"].float().norm()))
    return layer, x, logits, bias, y, saved, dy, grads


if __name__ == "__main__":
    main()
