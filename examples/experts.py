"""A layer of experts: tokens routed to gated feed-forward blocks, trained in 16 bits, served in
E4M3, with low-rank adapters beside its output projection.

    y[t] = sum_j w[t, j] E_{ids[t, j]}(x[t]),   E_e(x) = act(x Wg_e^T) * (x Wu_e^T)
    z[t] = y[t] Wo^T + scale_a (y[t] A_a^T) B_a^T,   a the adapter of token t's request

Training: route_contiguous and dispatch_f16 bring the tokens into segments, gated_f16 runs each
expert on its segment, combine_f16 brings the results back; the gradients go the same way in
reverse.  Serving: the same layer with dispatch_fp8 and grouped_fp8_masked, whose sizes no host
has to know, and lora_f16 beside gemm_f16.

    python examples/experts.py [--tokens 512] [--experts 8] [--choices 2] [--hidden 512] [--inter 256]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fine_grained_fp8_persistent_gb300 as fg  # noqa: E402


def choose(logits, choices):
    """The experts of each token and their weights: a softmax over the chosen logits."""
    top = torch.topk(logits, choices, dim=1)
    return top.indices, torch.softmax(top.values.float(), dim=1)


def forward(x, ids, w, wg, wu, act="silu"):
    """The layer's output and what its gradients need.  wg, wu: (experts, inter, hidden)."""
    route = fg.route_contiguous(ids, wg.shape[0])
    xs = fg.dispatch_f16(x, route)
    starts = route.starts.tolist()                        # the segments are the host's loop here
    ys = torch.empty(xs.shape[0], wg.shape[1], dtype=x.dtype, device=x.device)
    kept = []
    for e in range(wg.shape[0]):
        rows = slice(starts[e], starts[e + 1])
        ys[rows], g, u = fg.gated_f16(xs[rows], wg[e], wu[e], act, save=True)
        kept.append((rows, g, u))
    return fg.combine_f16(ys, w, route), (route, xs, ys, kept)


def backward(dy, w, wg, wu, saved, act="silu"):
    """Gradients of x, w, wg and wu."""
    route, xs, ys, kept = saved
    dys, dw = fg.combine_f16_backward(dy, ys, w, route)
    dxs = torch.empty_like(xs)
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
    for e, (rows, g, u) in enumerate(kept):
        dxs[rows], dwg[e], dwu[e] = fg.gated_f16_backward(dys[rows], xs[rows], wg[e], wu[e], g, u, act)
    return fg.dispatch_f16_backward(dxs, route), dw, dwg, dwu


class Server:
    """The layer with E4M3 weights: slots for `most` tokens per expert, no size read back."""

    def __init__(self, wg, wu, most, fmt="ue8m0"):
        self.fmt, self.most, self.experts = fmt, most, wg.shape[0]
        self.gate, self.up = (fg.quantize_128x128(w, fmt) for w in (wg, wu))

    def __call__(self, x, ids, w):
        route = fg.route_masked(ids, self.experts, self.most)
        xq, sfa = fg.dispatch_fp8(x, route, self.fmt)
        g, u = (fg.grouped_fp8_masked(xq, sfa, *weight, route.counts, self.fmt) for weight in (self.gate, self.up))
        return fg.combine_f16(torch.nn.functional.silu(g) * u, w, route)


def project(y, wo, a, b, scale, adapters):
    """y Wo^T with the adapter of each token's request beside it (-1: none)."""
    route = fg.route_contiguous(adapters, a.shape[0], align=16)
    z = fg.gemm_f16(y, wo)
    return fg.lora_f16(y, a, b, route, scale=scale, base=z, out=z)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--choices", type=int, default=2)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--inter", type=int, default=256)
    ap.add_argument("--steps", type=int, default=10)
    o = ap.parse_args(argv)
    gen = torch.Generator(device="cuda:0").manual_seed(0)

    def normal(*shape):
        return (torch.randn(*shape, generator=gen, device="cuda:0") / shape[-1] ** 0.5).bfloat16()
    x = torch.randn(o.tokens, o.hidden, generator=gen, device="cuda:0").bfloat16()
    router, wg, wu = normal(o.experts, o.hidden), normal(o.experts, o.inter, o.hidden), normal(o.experts, o.inter, o.hidden)
    want = forward(x, *choose(x.float() @ normal(o.experts, o.hidden).float().t(), o.choices), normal(*wg.shape), normal(*wu.shape))[0].float()
    master = [t.float() for t in (router, wg, wu)]
    adam = torch.optim.Adam(master, lr=2e-3)
    for step in range(o.steps):
        r, g16, u16 = master[0].requires_grad_(), master[1].bfloat16(), master[2].bfloat16()
        ids, w = choose(x.float() @ r.t(), o.choices)
        y, saved = forward(x, ids, w.detach(), g16, u16)
        err = y.float() - want
        print(f"step {step}: loss {float((err * err).mean()):.5f}")
        _, dw, dwg, dwu = backward((err * (2.0 / err.numel())).bfloat16(), w.detach(), g16, u16, saved)
        adam.zero_grad()
        w.backward(dw)                                    # the router's gradient, through torch
        master[1].grad, master[2].grad = dwg.float(), dwu.float()
        adam.step()
    serve = Server(g16, u16, o.tokens)
    served = serve(x, ids, w.detach()).float()
    rel = float((served - y.float()).norm() / y.float().norm())
    print(f"served in E4M3: relative error {rel:.3f}")
    adapters = torch.randint(-1, 4, (o.tokens,), generator=gen, device="cuda:0")
    z = project(y, normal(o.hidden, o.inter), normal(4, 16, o.inter), normal(4, o.hidden, 16), None, adapters)
    print(f"projected with adapters: {tuple(z.shape)}")
    return rel


if __name__ == "__main__":
    main()
