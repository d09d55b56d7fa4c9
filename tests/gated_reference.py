"""Plain 64-bit forms of the gated and 4-bit matrix-vector operators, with bounds on
how far a kernel may be off, derived from how it may compute.

Rounding model.  R is the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 fp16) and
T half its smallest subnormal.  A product of K terms is accumulated in FP32 by steps of
16 terms, each of which may drop 2^-23 of the running magnitude, and a few more joins:
gamma(K) = (K / 16 + 32) 2^-23 of sum |a||b|.  The activation and its slope are within
E = 2^-19 of a g-sized (unit-sized) value.  Slopes are at most 1.13 in magnitude.
"""
from __future__ import annotations

import math

import torch

GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715
ACTS = ("silu", "gelu_tanh")
E = 2.0 ** -19
SLOPE = 1.13


def unit(dtype) -> tuple[float, float]:
    return (2.0 ** -8, 2.0 ** -134) if dtype == torch.bfloat16 else (2.0 ** -11, 2.0 ** -25)


def gamma(K: int) -> float:
    return (K / 16 + 32) * 2.0 ** -23


def act64(g, act):
    y = g if act == "silu" else 2.0 * GELU_A * (g + GELU_B * g ** 3)
    return g * torch.sigmoid(y)


def slope64(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return s + g * s * (1.0 - s)
    s = torch.sigmoid(2.0 * GELU_A * (g + GELU_B * g ** 3))
    return s + g * s * (1.0 - s) * 2.0 * GELU_A * (1.0 + 3.0 * GELU_B * g ** 2)


def project64(x, w):
    """X W^T in 64 bits and the bound on an FP32-accumulated one."""
    x, w = x.double(), w.double()
    return x @ w.t(), gamma(x.shape[1]) * (x.abs() @ w.abs().t())


def gate64(g, dg, u, du, act, dtype):
    """a(G) U and the bound on one taken from G, U that are off by dg, du and rounded once."""
    R, T = unit(dtype)
    a = act64(g, act)
    h = a * u
    da = SLOPE * dg + E * g.abs()
    err = da * u.abs() + a.abs() * du + da * du
    return h, err + R * (h.abs() + err) + T


def forward64(x, wg, wu, act):
    """(H, G, U) in 64 bits and a bound on each."""
    R, T = unit(x.dtype)
    g, dg = project64(x, wg)
    u, du = project64(x, wu)
    h, dh = gate64(g, dg, u, du, act, x.dtype)
    return (h, g, u), (dh, dg + R * (g.abs() + dg) + T, du + R * (u.abs() + du) + T)


def backward64(dh, x, wg, wu, g, u, act):
    """(dX, dWg, dWu) in 64 bits from the kept G, U, and a bound on each: dG and dU are
    rounded to the 16-bit type before the products."""
    R, T = unit(x.dtype)
    dh, x, wg, wu, g, u = (t.double() for t in (dh, x, wg, wu, g, u))
    dg, du = dh * u * slope64(g, act), dh * act64(g, act)
    ddg = R * dg.abs() + (1.0 + R) * 2.0 * E * (dh * u).abs() + T
    ddu = R * du.abs() + (1.0 + R) * 2.0 * E * (dh * g).abs() + T
    dx, dwg, dwu = dg @ wg + du @ wu, dg.t() @ x, du.t() @ x

    def bound(value, err, mags, terms):
        err = err + gamma(terms) * mags
        return err + R * (value.abs() + err) + T

    gm, um = dg.abs() + ddg, du.abs() + ddu
    return (dx, dwg, dwu), (
        bound(dx, ddg @ wg.abs() + ddu @ wu.abs(), gm @ wg.abs() + um @ wu.abs(), 2 * wg.shape[0]),
        bound(dwg, ddg.t() @ x.abs(), gm.t() @ x.abs(), x.shape[0]),
        bound(dwu, ddu.t() @ x.abs(), um.t() @ x.abs(), x.shape[0]))


def gemv64(x, w64):
    """X W^T and the bound on a matrix-vector kernel's: FP32 sums, and rows of X that may be
    scaled by a power of two into fp16 (what is below 2^-32 of the row's largest |x| then
    rounds by up to 2^-40 of it)."""
    x = x.double()
    w = w64.to(x.device)
    y = x @ w.t()
    err = gamma(x.shape[1]) * (x.abs() @ w.abs().t())
    if x.shape[0] and x.shape[1]:
        err = err + 2.0 ** -40 * x.abs().amax(1, keepdim=True) * w.abs().sum(1)
    return y, err


def close(got, want, bound, what=""):
    g = got.double()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    if got.dtype == torch.float16:
        # past the type's range (what rounds above 65504) the result is infinite; a value whose
        # bound reaches across the edge may be either
        edge = 65520.0
        past = want.abs() - bound >= edge
        assert torch.equal(g[past], torch.copysign(torch.full_like(want[past], torch.inf), want[past])), what
        inside = want.abs() + bound < edge
        g, want, bound = g[inside], want[inside], bound[inside]
        if not g.numel():
            return
    assert torch.isfinite(g).all(), f"{what}: non-finite values"
    over = (g - want).abs() - bound
    assert not (over > 0).any(), (f"{what}: {int((over > 0).sum())} of {over.numel()} outside the bound, worst by "
                                  f"{float(over.max()):.3e} at {int(over.argmax())}")
