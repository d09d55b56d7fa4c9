"""Plain forms of the operators whose rows choose their own weights: the routing by a walk over
the ids, the rest in 64 bits with bounds on how far a kernel may be off, derived from how it
may compute.  R is the unit roundoff of the 16-bit type, T half its smallest subnormal
(gated_reference.unit); F = 2^-24 is that of FP32.
"""
from __future__ import annotations

import numpy as np
import torch

from gated_reference import gamma, unit

F = 2.0 ** -24


def route(ids, G, align, M=None, slots=0):
    """(rows, src, m_indices, counts, starts) as int32 numpy arrays, entry by entry."""
    flat = np.asarray(ids).reshape(-1)
    counts = np.zeros(G, np.int64)
    rank = np.full(flat.size, -1, np.int64)
    for i, g in enumerate(flat):
        if 0 <= g < G:
            rank[i] = counts[g]
            counts[g] += 1
    if slots:
        starts = np.arange(G + 1) * slots
        counts = np.minimum(counts, slots)
    else:
        starts = np.concatenate(([0], np.cumsum(-(-counts // align) * align)))
    M = int(starts[-1]) if M is None else M
    rows = np.full(flat.size, -1, np.int32)
    src, m_indices = np.full(M, -1, np.int32), np.full(M, -1, np.int32)
    for i, g in enumerate(flat):
        if rank[i] >= 0 and (not slots or rank[i] < slots):
            rows[i] = starts[g] + rank[i]
            src[rows[i]], m_indices[rows[i]] = i, g
    return rows.reshape(np.asarray(ids).shape), src, m_indices, counts.astype(np.int32), starts.astype(np.int32)


def random_ids(T, k, G, seed, absent=0.0, skew=0.0):
    """int32 CPU ids with replacement (a group may stand twice in a token's list); `skew` of them
    in group 0, `absent` of them -1."""
    gen = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, G, (T, k), generator=gen, dtype=torch.int32)
    if skew:
        ids[torch.rand(T, k, generator=gen) < skew] = 0
    if absent:
        ids[torch.rand(T, k, generator=gen) < absent] = -1
    return ids


def rounded(value, err, dtype):
    """The bound on a value that is off by err in FP32 and then rounded to dtype."""
    R, T = unit(dtype)
    return err + R * (value.abs() + err) + T


def combine64(ys, w, rows, dtype):
    """Y and its bound: k FP32 products and sums, one rounding."""
    ok = (rows >= 0).unsqueeze(-1)
    y = torch.where(ok, ys.double()[rows.clamp(min=0).long()], 0.0)
    ww = torch.ones(rows.shape, dtype=torch.float64, device=ys.device) if w is None else torch.where(rows >= 0, w.double(), 0.0)
    terms = ww.unsqueeze(-1) * y
    value = terms.sum(1)
    return value, rounded(value, (rows.shape[1] + 1) * F * terms.abs().sum(1), dtype)


def combine_backward64(dy, ys, w, rows, M, dtype):
    """(dYs, dw) and their bounds.  A dot product's longest chain: a thread's products (8 for each
    256 pieces of 8), five steps over lanes, eight over warps."""
    T, N = dy.shape
    d = dy.double()
    dys = torch.zeros((M, N), dtype=torch.float64, device=dy.device)
    dw = torch.zeros(rows.shape, dtype=torch.float64, device=dy.device)
    mag = torch.zeros_like(dw)
    for j in range(rows.shape[1]):
        has = torch.nonzero(rows[:, j] >= 0).view(-1)
        at = rows[has, j].long()
        dys[at] = w[has, j].double().unsqueeze(1) * d[has]
        y = ys.double()[at]
        dw[has, j] = (d[has] * y).sum(1)
        mag[has, j] = (d[has].abs() * y.abs()).sum(1)
    chain = 8 * -(-N // 2048) + 13
    return (dys, dw), (rounded(dys, F * dys.abs(), dtype), chain * F * mag + F * dw.abs() + 2.0 ** -149)


def lora64(x, a, b, ids, scale, base):
    """out and its bound.  X A^T and P B^T accumulate in FP32 (gamma; 64 sums more over warps and
    CTAs); P is scaled (one rounding) and split in two 16-bit values, which leaves R^2 of it, and
    in fp16 2^-39 of its row's largest (the rest of a small one below the type's subnormals)."""
    dtype = x.dtype
    R, _ = unit(dtype)
    T, N = x.shape[0], b.shape[1]
    out = torch.zeros((T, N), dtype=torch.float64, device=x.device) if base is None else base.double().clone()
    err = F * out.abs()
    ids = ids.view(-1)
    for g in range(a.shape[0]):
        mine = torch.nonzero(ids == g).view(-1)
        if not len(mine):
            continue
        s = 1.0 if scale is None else float(scale[g])
        xg, ag, bg = x[mine].double(), a[g].double(), b[g].double()
        p = s * (xg @ ag.t())
        ep = abs(s) * (gamma(x.shape[1]) + 64 * F) * (xg.abs() @ ag.abs().t()) + F * p.abs()
        ep = ep + R * R * (p.abs() + ep) + 2.0 ** -39 * (p.abs() + ep).amax(1, keepdim=True)
        d = p @ bg.t()
        ed = ep @ bg.abs().t() + gamma(2 * a.shape[1]) * ((p.abs() + ep) @ bg.abs().t())
        out[mine] += d
        err[mine] += ed + F * (d.abs() + out[mine].abs())
    return out, rounded(out, err, dtype)
