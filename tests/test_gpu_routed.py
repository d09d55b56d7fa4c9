"""GPU tests of the routing, dispatch and combine operators and their gradients: the routing
against a walk over the ids, copies bit by bit, sums against their definition in 64 bits."""
import numpy as np
import pytest
import torch

import gated_reference
import routed_reference as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]
FMTS = [0, 1]


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def _same(route, want, what=""):
    for got, w, name in zip((route.rows, route.src, route.m_indices, route.counts, route.starts), want, route._fields):
        if got is not None:
            assert np.array_equal(got.cpu().numpy(), w), (what, name)


# ----------------------------------------------------------------- routing
# no tokens, one, lists of each form (test_gpu_routed_edges.py stands on their borders), more groups
# than entries, every group of 1024, ids that fill no step of 32
ROUTES = [(0, 1, 4), (1, 1, 1), (1, 8, 8), (5, 3, 7), (33, 2, 5), (1000, 1, 1), (4096, 1, 64), (4097, 1, 3), (512, 8, 256),
          (513, 8, 256), (700, 9, 1000), (20000, 4, 1024), (3, 40, 6)]


@pytest.mark.parametrize("int64", [False, True])
@pytest.mark.parametrize("T,k,G", ROUTES)
def test_route_contiguous(fg, dev, T, k, G, int64):
    for align, absent, skew in [(128, 0.0, 0.0), (16, 0.2, 0.5), (1, 0.9, 0.0), (100, 0.0, 1.0), (128, 1.0, 0.0)]:
        ids = ref.random_ids(T, k, G, T + k + G, absent, skew)
        r = fg.route_contiguous((ids.long() if int64 else ids).to(dev), G, align)
        M = fg.route_rows(T, k, G, align)
        assert r.src.shape == (M,) and M % align == 0
        _same(r, ref.route(ids.numpy(), G, align, M), (align, absent, skew))
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("T,k,G", ROUTES)
def test_route_masked(fg, dev, T, k, G):
    for Mmax, absent, skew in [(256, 0.0, 0.0), (1, 0.2, 0.5), (7, 0.0, 0.3)]:
        ids = ref.random_ids(T, k, G, T + k + G + 1, absent, skew)
        r = fg.route_masked(ids.to(dev), G, Mmax)
        want = ref.route(ids.numpy(), G, 1, G * Mmax, Mmax)
        _same(r, want, (Mmax, absent, skew))
        assert r.counts.max() <= Mmax
    assert fg.check_status()[0] == 0


def test_route_of_a_long_list(fg, dev):
    T, k, G = 150000, 8, 300
    ids = ref.random_ids(T, k, G, 3, 0.01, 0.2)
    r = fg.route_contiguous(ids.to(dev), G)
    flat = ids.view(-1).numpy()
    order = np.argsort(np.where(flat < 0, G, flat), kind="stable")
    counts = np.bincount(flat[flat >= 0], minlength=G)
    starts = np.concatenate(([0], np.cumsum(-(-counts // 128) * 128)))
    rows = np.full(flat.size, -1)
    at = 0
    for g in range(G):
        rows[order[at:at + counts[g]]] = starts[g] + np.arange(counts[g])
        at += counts[g]
    assert np.array_equal(r.rows.cpu().numpy().reshape(-1), rows)
    assert np.array_equal(r.starts.cpu().numpy(), starts) and np.array_equal(r.counts.cpu().numpy(), counts)
    src = np.full(r.src.shape[0], -1)
    src[rows[rows >= 0]] = np.flatnonzero(rows >= 0)
    assert np.array_equal(r.src.cpu().numpy(), src)
    assert np.array_equal(r.m_indices.cpu().numpy(), np.where(src < 0, -1, flat[src.clip(0)]))


def test_route_more_rows_than_needed(fg, dev):
    ids = ref.random_ids(40, 2, 5, 1, 0.1)
    r = fg.route_contiguous(ids.to(dev), 5, 128, M=2048)
    _same(r, ref.route(ids.numpy(), 5, 128, 2048))


@pytest.mark.parametrize("value", [5, -2, 1 << 20, -(1 << 31)])
def test_ids_out_of_range_are_reported(fg, dev, value):
    ids = ref.random_ids(50, 2, 5, 1)
    bad = ids.clone()
    bad[17, 1] = value
    ids[17, 1] = -1
    r = fg.route_contiguous(bad.to(dev), 5)
    assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT
    _same(r, ref.route(ids.numpy(), 5, 128, fg.route_rows(50, 2, 5)))
    assert fg.check_status()[0] == 0
    big = ids.long()
    big[17, 1] = (1 << 32) + 3                       # in range only in its low half
    r = fg.route_masked(big.to(dev), 5, 64)
    assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT
    _same(r, ref.route(ids.numpy(), 5, 1, 320, 64))


# ----------------------------------------------------------------- dispatch
# (T, k, G, H): no token, one, rows of one 16-byte piece, rows that fill no item, many choices
CASES = [(0, 2, 3, 64), (1, 1, 1, 8), (1, 8, 32, 7168), (7, 3, 5, 72), (64, 2, 9, 1032), (129, 4, 3, 1800), (40, 33, 4, 136),
         (300, 6, 70, 520), (2, 70, 8, 2056)]


def _bits(T, H, seed, dev):
    """Any bits at all, NaN payloads among them."""
    gen = torch.Generator().manual_seed(seed)
    return torch.randint(-32768, 32768, (T, H), generator=gen, dtype=torch.int32).to(torch.int16).to(dev).view(torch.bfloat16)


@pytest.mark.parametrize("absent", [0.0, 0.4])
@pytest.mark.parametrize("T,k,G,H", CASES)
def test_dispatch_f16(fg, dev, T, k, G, H, absent):
    ids = ref.random_ids(T, k, G, 7, absent)
    x = _bits(T, H, 8, dev)
    r = fg.route_contiguous(ids.to(dev), G)
    xs = fg.dispatch_f16(x, r, out=_bits(r.src.shape[0], H, 9, dev))
    rows, src = r.rows.cpu(), r.src.cpu()
    want = torch.zeros(src.shape[0], H, dtype=torch.int16)
    own = src >= 0
    want[own] = x.view(torch.int16).cpu()[(src[own] // k).long()]
    assert torch.equal(xs.view(torch.int16).cpu(), want)
    # masked: rows without an entry stay as they are
    m = fg.route_masked(ids.to(dev), G, 5)
    before = _bits(5 * G, H, 10, dev)
    xs = fg.dispatch_f16(x, m, out=before.clone())
    src = m.src.cpu()
    want = before.view(torch.int16).cpu().clone()
    want[src >= 0] = x.view(torch.int16).cpu()[(src[src >= 0] // k).long()]
    assert torch.equal(xs.view(torch.int16).cpu(), want)
    assert torch.equal(fg.dispatch_f16(x.view(torch.float16), r).view(torch.int16), fg.dispatch_f16(x, r).view(torch.int16))
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,k,G,K", [(1, 1, 1, 128), (1, 8, 32, 7168), (5, 3, 4, 640), (77, 2, 9, 1152), (300, 6, 70, 512), (3, 40, 5, 256)])
def test_dispatch_fp8_gives_the_bits_of_quantize(fg, dev, T, k, G, K, fmt):
    ids = ref.random_ids(T, k, G, 17, 0.2)
    gen = torch.Generator().manual_seed(18)
    x = torch.randn(T, K, generator=gen)
    x *= torch.exp2(torch.randint(-30, 30, (T, K // 128, 1), generator=gen).float()).expand(T, K // 128, 128).reshape(T, K)
    x[0, :128] = 0.0
    x[-1, -128:] = 1e-39                                    # subnormal scales
    x = x.bfloat16().to(dev)
    codes, table = (t.cpu() for t in fg.quantize_1x128(x, fmt))
    for r in (fg.route_contiguous(ids.to(dev), G), fg.route_masked(ids.to(dev), G, 7)):
        M, slots = r.src.shape[0], r.slots
        shape = fg.sfa_shape(slots or M, K, fmt)[0]
        xq = torch.full((M, K), 0x5A, dtype=torch.uint8, device=dev)
        sfa = torch.full((G, *shape) if slots else shape, 7, dtype=torch.float32 if fmt == 0 else torch.int32, device=dev)
        fg.dispatch_fp8(x, r, fmt, xq=xq, sfa=sfa)
        src = r.src.cpu().long()
        own = torch.nonzero(src >= 0).view(-1)
        want_q = torch.full((M, K), 0x5A, dtype=torch.uint8)
        want_q[own] = codes[src[own] // k]
        want_s = torch.full(tuple(sfa.shape), 7, dtype=sfa.dtype)
        per_token = table[:, :T].t()
        if slots:
            want_s[own // slots, :, own % slots] = per_token[src[own] // k]
        else:
            want_s[:, own] = per_token[src[own] // k].t()
        assert torch.equal(xq.cpu(), want_q)
        assert torch.equal(sfa.cpu().view(torch.int32), want_s.view(torch.int32))
    assert fg.check_status()[0] == 0


# ----------------------------------------------------------------- combine and gradients
def _routed(fg, dev, T, k, G, H, dtype, absent, masked, seed=0):
    ids = ref.random_ids(T, k, G, 27 + seed, absent, 0.2)
    r = fg.route_masked(ids.to(dev), G, max(1, T * k // G)) if masked else fg.route_contiguous(ids.to(dev), G)
    gen = torch.Generator().manual_seed(28 + seed)
    ys = torch.randn(r.src.shape[0], H, generator=gen).to(dtype).to(dev)
    ys[r.src < 0] = float("nan")                            # rows without an entry are never looked at
    w = torch.randn(T, k, generator=gen).to(dev)
    return r, ys, w, gen


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,G,H", CASES)
def test_combine(fg, dev, T, k, G, H, dtype, masked):
    r, ys, w, _ = _routed(fg, dev, T, k, G, H, dtype, 0.3, masked)
    w[r.rows < 0] = float("nan")                            # nor their weights
    y = fg.combine_f16(ys, w, r)
    gated_reference.close(y, *ref.combine64(ys, w, r.rows, dtype))
    assert torch.equal(y, fg.combine_f16(ys, w, r))
    dx = fg.dispatch_f16_backward(ys, r)
    gated_reference.close(dx, *ref.combine64(ys, None, r.rows, dtype))
    assert torch.equal(dx, fg.combine_f16(ys, None, r))
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,G,H", CASES)
def test_combine_backward(fg, dev, T, k, G, H, dtype, masked):
    r, ys, w, gen = _routed(fg, dev, T, k, G, H, dtype, 0.3, masked)
    w[r.rows < 0] = float("nan")
    dy = torch.randn(T, H, generator=gen).to(dtype).to(dev)
    out = torch.full_like(ys, 3.0)
    dys, dw = fg.combine_f16_backward(dy, ys, w, r, dys=out)
    (want_y, want_w), (by, bw) = ref.combine_backward64(dy, ys, w, r.rows, ys.shape[0], dtype)
    if masked:
        assert (dys[r.src < 0] == 3.0).all()
        dys, want_y, by = dys[r.src >= 0], want_y[r.src >= 0], by[r.src >= 0]
    gated_reference.close(dys, want_y, by, "dys")
    gated_reference.close(dw, want_w, bw, "dw")
    assert torch.equal(dw, fg.combine_f16_backward(dy, ys, w, r)[1])
    assert fg.check_status()[0] == 0


def test_gradients_against_differences(fg, dev):
    """dys and dw along random directions against central differences of sum(dY * Y) in 64 bits
    (Y is linear in each, so a difference has no error of its own but FP64's)."""
    T, k, G, H = 9, 3, 4, 40
    r, ys, w, gen = _routed(fg, dev, T, k, G, H, torch.float16, 0.2, False)
    ys = torch.nan_to_num(ys)
    dy = torch.randn(T, H, generator=gen).half().to(dev)
    dys, dw = fg.combine_f16_backward(dy, ys, w, r)
    (_, _), (by, bw) = ref.combine_backward64(dy, ys, w, r.rows, ys.shape[0], torch.float16)
    dxs = torch.randn(ys.shape, generator=gen).half().to(dev)
    dx = fg.dispatch_f16_backward(dxs, r)
    bx = ref.combine64(dxs, None, r.rows, torch.float16)[1]

    def loss(y, ww):
        at = r.rows.clamp(min=0).long()
        return ((r.rows >= 0).unsqueeze(-1) * ww.unsqueeze(-1) * y[at]).sum(1).mul(dy.double()).sum()

    def way_in(x):
        src = r.src.long()
        return torch.where((src >= 0).unsqueeze(-1), x[src.clamp(min=0) // k], 0.0).mul(dxs.double()).sum()
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        vy, vw = (torch.randn(t.shape, generator=g, dtype=torch.float64).to(dev) for t in (ys, w))
        vx = torch.randn(T, H, generator=g, dtype=torch.float64).to(dev)
        y64, w64, e = ys.double(), w.double(), 1e-3
        slope = float(loss(y64 + e * vy, w64) - loss(y64 - e * vy, w64)) / (2 * e)
        assert abs(slope - float((dys.double() * vy).sum())) <= float((by * vy.abs()).sum()) + 1e-9 * abs(slope) + 1e-9
        slope = float(loss(y64, w64 + e * vw) - loss(y64, w64 - e * vw)) / (2 * e)
        assert abs(slope - float((dw.double() * vw).sum())) <= float((bw * vw.abs()).sum()) + 1e-9 * abs(slope) + 1e-9
        slope = float(way_in(e * vx) - way_in(-e * vx)) / (2 * e)
        assert abs(slope - float((dx.double() * vx).sum())) <= float((bx * vx.abs()).sum()) + 1e-9 * abs(slope) + 1e-9


def test_infinities_and_nans_stay_in_their_tokens(fg, dev):
    r, ys, w, gen = _routed(fg, dev, 20, 2, 4, 64, torch.bfloat16, 0.0, False)
    ys[r.rows[3, 1].long()] = float("inf")
    ys[r.rows[7, 0].long(), 5] = float("nan")
    w[11, 0] = float("nan")
    y = fg.combine_f16(ys, w, r)
    assert torch.isinf(y[3]).all() and torch.isnan(y[7, 5]) and torch.isnan(y[11]).all()
    fine = torch.ones(20, 64, dtype=torch.bool, device=dev)
    fine[[3, 11]] = False
    fine[7, 5] = False
    assert torch.isfinite(y[fine]).all()
    w[11, 0] = 0.0                                          # a weight of zero takes part: 0 * inf
    ys[r.rows[11, 0].long()] = float("inf")
    assert torch.isnan(fg.combine_f16(ys, w, r)[11]).all()


def test_rows_out_of_range_are_reported(fg, dev):
    """They count as no row: nothing outside the layout is read or written."""
    r, ys, w, gen = _routed(fg, dev, 30, 2, 4, 64, torch.bfloat16, 0.0, False)
    M = ys.shape[0]
    good, bad = r.rows.clone(), r.rows.clone()
    for i, v in ((3, M), (9, -2), (15, 2 ** 31 - 1)):
        good[i, 1], bad[i, 1] = -1, v
    dy, x = (torch.randn(30, 64, generator=gen).bfloat16().to(dev) for _ in range(2))
    calls = [lambda q: fg.combine_f16(ys, w, q), lambda q: fg.dispatch_f16(x, q), lambda q: fg.dispatch_f16_backward(ys, q),
             lambda q: torch.cat([t.float().flatten() for t in fg.combine_f16_backward(dy, ys, w, q)])]
    # of the rows that lost their entry the layout's src still says that they have one
    lost = r.rows[good < 0].long()
    for i, call in enumerate(calls):
        a = call(r._replace(rows=good))
        assert fg.check_status()[0] == 0
        b = call(r._replace(rows=bad))
        assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT
        if i == 1:
            a[lost] = b[lost] = 0
        if i == 3:
            a[: M * 64].view(M, 64)[lost] = 0
            b[: M * 64].view(M, 64)[lost] = 0
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)), i


# ----------------------------------------------------------------- together
def _expert_weights(fg, dev, G, N, K, fmt, seed):
    gen = torch.Generator().manual_seed(seed)
    w = (torch.randn(G, N, K, generator=gen) / K ** 0.5).bfloat16().to(dev)
    return w, fg.quantize_128x128(w, fmt)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("fmt", FMTS)
def test_expert_layer(fg, dev, fmt, masked):
    """Routing, dispatch with quantization, the grouped product, combine: against the product of
    the same quantized operands token by token in 64 bits.  The product may be off by FP32
    accumulation (gamma) and its rounding to bf16, which combine carries on."""
    T, k, G, K, N = 150, 3, 5, 384, 256
    ids = ref.random_ids(T, k, G, 5, 0.1)
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(T, K, generator=gen).bfloat16().to(dev)
    wt = torch.rand(T, k, generator=gen).to(dev)
    w, (wq, sfb) = _expert_weights(fg, dev, G, N, K, fmt, 7)
    if masked:
        r = fg.route_masked(ids.to(dev), G, 128)
        xq, sfa = fg.dispatch_fp8(x, r, fmt)
        ys = fg.grouped_fp8_masked(xq, sfa, wq, sfb, r.counts, fmt)
    else:
        r = fg.route_contiguous(ids.to(dev), G)
        xq, sfa = fg.dispatch_fp8(x, r, fmt)
        ys = fg.grouped_fp8_contiguous(xq, sfa, wq, sfb, r.m_indices, fmt)
    y = fg.combine_f16(ys, wt, r)
    assert fg.check_status()[0] == 0
    # the same operands back in 64 bits
    q, s = fg.quantize_1x128(x, fmt)
    if fmt == 0:
        sx = s[:, :T].t().double()
        sw = sfb.double().repeat_interleave(128, 1)[:, :N]
    else:
        e = s.view(torch.uint8).view(s.shape[0], s.shape[1], 4)[:, :T].permute(1, 0, 2).reshape(T, -1)[:, : K // 128]
        sx = torch.exp2(e.double() - 127)
        e = sfb.view(torch.uint8).view(G, sfb.shape[1], sfb.shape[2], 4)[:, :, :N].permute(0, 2, 1, 3).reshape(G, N, -1)[..., : K // 128]
        sw = torch.exp2(e.double() - 127)
    xd = (q.view(torch.float8_e4m3fn).double().view(T, -1, 128) * sx.unsqueeze(-1)).view(T, K)
    wd = (wq.view(torch.float8_e4m3fn).double().view(G, N, -1, 128) * sw.unsqueeze(-1)).view(G, N, K)
    R, _ = gated_reference.unit(torch.bfloat16)
    want, err = torch.zeros(T, N, dtype=torch.float64, device=dev), torch.zeros(T, N, dtype=torch.float64, device=dev)
    mag = torch.zeros_like(want)
    for j in range(k):
        for g in range(G):
            mine = torch.nonzero((ids[:, j].to(dev) == g) & (r.rows[:, j] >= 0)).view(-1)
            p, a = xd[mine] @ wd[g].t(), xd[mine].abs() @ wd[g].abs().t()
            ww = wt[mine, j].double().unsqueeze(1)
            want[mine] += ww * p
            ep = gated_reference.gamma(K) * a
            err[mine] += ww * (ep + R * (p.abs() + ep))
            mag[mine] += ww * p.abs()
    gated_reference.close(y, want, ref.rounded(want, err + (k + 1) * ref.F * (mag + err), torch.bfloat16))


def test_training_layer(fg, dev):
    """Dispatch, each expert's gated block over its segment, combine, and all gradients: dX, dw and
    the experts' against 64-bit autograd of the same layer, which rounds nowhere.  Each of the
    five 16-bit roundings on the way (H, G and U, dYs, dG and dU, dXs) is at most R of its
    value, so the whole is off by a few R of the magnitudes that meet; 8 R of the largest
    value of each gradient holds it."""
    T, k, G, K, N = 96, 2, 3, 64, 48
    ids = ref.random_ids(T, k, G, 11, 0.1)
    gen = torch.Generator().manual_seed(12)
    x = torch.randn(T, K, generator=gen).half().to(dev)
    wt = torch.rand(T, k, generator=gen).to(dev)
    wg, wu = ((torch.randn(G, N, K, generator=gen) / K ** 0.5).half().to(dev) for _ in range(2))
    dy = torch.randn(T, N, generator=gen).half().to(dev)
    r = fg.route_contiguous(ids.to(dev), G)
    xs = fg.dispatch_f16(x, r)
    ys = torch.zeros(xs.shape[0], N, dtype=x.dtype, device=dev)
    starts, kept = r.starts.tolist(), []
    for g in range(G):
        s = slice(starts[g], starts[g + 1])
        ys[s], *gu = fg.gated_f16(xs[s], wg[g], wu[g], save=True)
        kept.append(gu)
    y = fg.combine_f16(ys, wt, r)
    dys, dw = fg.combine_f16_backward(dy, ys, wt, r)
    dxs = torch.zeros_like(xs)
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
    for g in range(G):
        s = slice(starts[g], starts[g + 1])
        dxs[s], dwg[g], dwu[g] = fg.gated_f16_backward(dys[s], xs[s], wg[g], wu[g], *kept[g])
    dx = fg.dispatch_f16_backward(dxs, r)
    assert fg.check_status()[0] == 0
    leaves = [t.double().requires_grad_() for t in (x, wt, wg, wu)]
    x64, w64, g64, u64 = leaves
    y64 = torch.zeros(T, N, dtype=torch.float64, device=dev)
    for j in range(k):
        for g in range(G):
            mine = torch.nonzero(ids[:, j].to(dev) == g).view(-1)
            a = x64[mine] @ g64[g].t()
            y64 = y64.index_add(0, mine, w64[mine, j].unsqueeze(1) * a * torch.sigmoid(a) * (x64[mine] @ u64[g].t()))
    y64.backward(dy.double())
    R, _ = gated_reference.unit(torch.float16)
    for got, want, what in ((y, y64.detach(), "y"), (dx, x64.grad, "dx"), (dw, w64.grad, "dw"), (dwg, g64.grad, "dwg"), (dwu, u64.grad, "dwu")):
        assert float((got.double() - want).abs().max()) <= 8 * R * float(want.abs().max()), what


def test_outputs_stay_inside_their_buffers(fg, dev):
    """Outputs at the front of larger buffers: nothing past their end is written."""
    T, k, G, H = 37, 3, 5, 136
    ids = ref.random_ids(T, k, G, 3, 0.2).to(dev)
    r = fg.route_contiguous(ids, G)
    M = r.src.shape[0]
    x, w = torch.randn(T, H, device=dev).bfloat16(), torch.rand(T, k, device=dev)

    def room(*shape, dtype=torch.bfloat16):
        n = int(np.prod(shape))
        buf = torch.full((n + 4096,), 7, dtype=dtype, device=dev)
        return buf, buf[:n].view(shape), n
    bufs = [room(M, H), room(T, H), room(T, H), room(M, H), room(T, k, dtype=torch.float32)]
    fg.dispatch_f16(x, r, out=bufs[0][1])
    fg.combine_f16(bufs[0][1], w, r, out=bufs[1][1])
    fg.dispatch_f16_backward(bufs[0][1], r, out=bufs[2][1])
    fg.combine_f16_backward(x, bufs[0][1], w, r, dys=bufs[3][1], dw=bufs[4][1])
    torch.cuda.synchronize()
    for buf, _, n in bufs:
        assert (buf[n:] == 7).all()


def test_streams_and_graphs(fg, dev):
    """On another stream than the current one, and captured once and replayed on other inputs."""
    T, k, G, H = 70, 2, 6, 256
    side = torch.cuda.Stream(dev)
    ids = ref.random_ids(T, k, G, 1, 0.1).to(dev)
    x, w = torch.randn(T, H, device=dev).bfloat16(), torch.rand(T, k, device=dev)

    def chain(stream=None):
        r = fg.route_contiguous(ids, G, stream=stream)
        xs = fg.dispatch_f16(x, r, stream=stream)
        xq, sfa = fg.dispatch_fp8(x, r, "ue8m0", stream=stream)
        y = fg.combine_f16(xs, w, r, stream=stream)
        dys, dw = fg.combine_f16_backward(y, xs, w, r, stream=stream)
        m = fg.route_masked(ids, G, 16, stream=stream)
        return [*r[:5], xs, y, dys, dw, fg.dispatch_f16_backward(dys, r, stream=stream), m.rows, m.src, m.counts], (xq, sfa, r)
    want, _ = chain()
    torch.cuda.synchronize()
    got, _ = chain(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held, _ = chain()
    for seed in (2, 3):
        ids.copy_(ref.random_ids(T, k, G, seed, 0.3))
        x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        want, _ = chain()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
    assert fg.check_status()[0] == 0


def test_long_list_in_a_graph(fg, dev):
    """A routing on a cluster of 16 CTAs, captured and replayed on other ids."""
    T, k, G = 9000, 4, 40
    ids = ref.random_ids(T, k, G, 1).to(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = fg.route_contiguous(ids, G)
    ids.copy_(ref.random_ids(T, k, G, 2, 0.2, 0.1))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held[:5], fg.route_contiguous(ids, G)[:5]))


def test_queue_of_dependent_calls(fg, dev):
    """Calls that each read what the one before wrote, with and without programmatic launches."""
    T, k, G, H = 500, 2, 8, 512
    ids = ref.random_ids(T, k, G, 1).to(dev)
    x = torch.randn(T, H, device=dev).bfloat16()
    half = torch.full((T, k), 0.5, device=dev)
    before = fg.set_pdl(True)
    try:
        for pdl in (True, False):
            fg.set_pdl(pdl)
            y = x
            for i in range(60):
                r = fg.route_contiguous(ids, G)
                y = fg.combine_f16(fg.dispatch_f16(y, r), half, r)
            assert torch.equal(y, x)                        # 0.5 x + 0.5 x, exact
    finally:
        fg.set_pdl(before)
    assert fg.check_status()[0] == 0
