"""A gated feed-forward block trained in 16 bits and served in 4.

    y = (act(x Wg^T) * (x Wu^T)) Wd^T

Training: gated_f16 (forward, keeping G and U), gemm_f16 (down projection and its
gradients) and gated_f16_backward; FP32 master weights and Adam in torch.  Serving: the three weights quantized once by quantize_fp4, one token at a time
through gated_gemv_fp4 and gemv_fp4.

    python examples/feed_forward.py [--tokens 512] [--hidden 1024] [--inter 2048] [--steps 20] [--fmt nvfp4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fine_grained_fp8_persistent_gb300 as fg  # noqa: E402


def forward(x, wg, wu, wd, act):
    h, g, u = fg.gated_f16(x, wg, wu, act, save=True)
    return fg.gemm_f16(h, wd), (h, g, u)


def backward(dy, x, wg, wu, wd, kept, act):
    h, g, u = kept
    dwd = fg.gemm_f16(dy.t().contiguous(), h.t().contiguous())       # dY^T H
    dh = fg.gemm_f16(dy, wd.t().contiguous())                        # dY Wd
    _, dwg, dwu = fg.gated_f16_backward(dh, x, wg, wu, g, u, act)
    return dwg, dwu, dwd


def train(tokens, hidden, inter, steps, act="silu", lr=2e-3, seed=0, device="cuda:0"):
    """Fits the block to another one of the same shape on a batch of tokens, with FP32 master
    weights and Adam; returns (losses, weights)."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def weights(scale):
        shapes = ((inter, hidden), (inter, hidden), (hidden, inter))
        return [torch.randn(s, generator=gen, device=device) * (scale / s[1] ** 0.5) for s in shapes]

    target = [w.bfloat16() for w in weights(1.0)]
    master = [w.float() + 0.3 * d for w, d in zip(target, weights(1.0))]
    adam = torch.optim.Adam(master, lr=lr, betas=(0.9, 0.95))
    x = torch.randn(tokens, hidden, generator=gen, device=device).bfloat16()
    want = forward(x, *target, act)[0].float()
    losses = []
    for _ in range(steps):
        wg, wu, wd = (w.bfloat16() for w in master)
        y, kept = forward(x, wg, wu, wd, act)
        err = y.float() - want
        losses.append(float((err * err).mean()))
        dy = (err * (2.0 / tokens)).bfloat16()                       # of the mean over tokens
        for w, d in zip(master, backward(dy, x, wg, wu, wd, kept, act)):
            w.grad = d.float()
        adam.step()
    return losses, [w.bfloat16() for w in master]


class Server:
    """The block with 4-bit weights, for a few tokens at a time."""

    def __init__(self, wg, wu, wd, fmt, act="silu"):
        self.fmt, self.act = fmt, act
        self.gate, self.up, self.down = (fg.quantize_fp4(w, fmt) for w in (wg, wu, wd))

    def __call__(self, x):
        h = fg.gated_gemv_fp4(x, *self.gate, *self.up, self.fmt, self.act)
        return fg.gemv_fp4(h, *self.down, self.fmt)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inter", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--act", default="silu", choices=["silu", "gelu_tanh"])
    ap.add_argument("--fmt", default="nvfp4", choices=["mxfp4", "nvfp4"])
    a = ap.parse_args(argv)
    losses, weights = train(a.tokens, a.hidden, a.inter, a.steps, a.act)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    serve = Server(*weights, a.fmt, a.act)
    x = torch.randn(8, a.hidden, device="cuda:0").bfloat16()
    full, _ = forward(x, *weights, a.act)
    one_by_one = torch.cat([serve(t[None]) for t in x])
    rel = float((one_by_one.float() - full.float()).norm() / full.float().norm())
    print(f"{a.fmt}: one token at a time, relative error against the 16-bit block {rel:.3f}")
    return losses, rel


if __name__ == "__main__":
    main()
