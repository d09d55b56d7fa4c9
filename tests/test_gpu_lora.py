"""GPU tests of lora_f16 against its definition in 64 bits."""
import pytest
import torch

import gated_reference
import routed_reference as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]
# (T, G, K, N, r): one token, one adapter, fewer tokens than adapters, sizes down to 8, ranks on both sides of each
# padded one, tokens that fill no tile, more tiles than SMs
SHAPES = [(1, 1, 8, 8, 8), (1, 4, 7168, 2048, 16), (2, 9, 40, 264, 24), (5, 3, 1032, 72, 32), (16, 2, 256, 128, 40), (17, 1, 512, 40, 64),
          (48, 64, 2056, 1800, 16), (33, 5, 136, 1000, 72), (70, 3, 200, 328, 128), (200, 7, 1024, 520, 8), (513, 6, 712, 1032, 48),
          (1500, 3, 264, 776, 64), (2600, 40, 520, 264, 16), (5000, 2, 136, 72, 104)]


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def _inputs(T, G, K, N, r, dtype, dev, absent=0.15, seed=0, skew=0.3):
    gen = torch.Generator().manual_seed(seed + T + K + N + r)
    x = torch.randn(T, K, generator=gen)
    x[:, :: max(1, K // 3)] *= 8.0
    a, b = torch.randn(G, r, K, generator=gen) / K ** 0.5, torch.randn(G, N, r, generator=gen) / r ** 0.5
    base = torch.randn(T, N, generator=gen)
    scale = torch.randn(G, generator=gen).to(dev)
    ids = ref.random_ids(T, 1, G, seed + T, absent, skew).view(-1).to(dev)
    return *(t.to(dtype).to(dev) for t in (x, a, b, base)), scale, ids


# rows of the routing and the form: tiles of 16 in segments of 16 and of 128 rows, blocks of 128
FORMS = [(16, 16), (128, 16), (128, 128)]


@pytest.mark.parametrize("align,rows", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,G,K,N,r", SHAPES)
def test_lora(fg, dev, monkeypatch, T, G, K, N, r, dtype, align, rows):
    x, a, b, base, scale, ids = _inputs(T, G, K, N, r, dtype, dev)
    route = fg.route_contiguous(ids, G, align)
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    out = fg.lora_f16(x, a, b, route, scale=scale, base=base)
    assert fg.last_tile().startswith("f16 lora ") and fg.last_tile().endswith(f"x{rows}")
    gated_reference.close(out, *ref.lora64(x, a, b, ids, scale, base))
    again = base.clone()
    assert fg.lora_f16(x, a, b, route, scale=scale, base=again, out=again) is again
    assert torch.equal(again, out)                          # in place, and run to run
    only = fg.lora_f16(x, a, b, route)
    gated_reference.close(only, *ref.lora64(x, a, b, ids, None, None))
    none = ids < 0
    assert torch.equal(out[none], base[none]) and not only[none].any()
    assert fg.check_status()[0] == 0


# 9000 tokens read adapters 567 times in tiles, in us: rank 32 21 against 26 in blocks, rank 64 30
# against 26
@pytest.mark.parametrize("T,r,form", [(100, 32, 16), (9000, 32, 16), (9000, 64, 128)])
def test_form_by_size(fg, dev, T, r, form):
    """Few tokens go in tiles whatever their segments, many of a large rank in blocks."""
    x, a, b, base, scale, ids = _inputs(T, 4, 1024, 1024, r, torch.bfloat16, dev)
    out = fg.lora_f16(x, a, b, fg.route_contiguous(ids, 4, 128), scale=scale, base=base)
    assert fg.last_tile().endswith(f"x{form}")
    gated_reference.close(out, *ref.lora64(x, a, b, ids, scale, base))


@pytest.mark.parametrize("align,rows", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
def test_no_token_has_an_adapter(fg, dev, monkeypatch, dtype, align, rows):
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    x, a, b, base, scale, ids = _inputs(40, 3, 64, 136, 16, dtype, dev)
    route = fg.route_contiguous(torch.full_like(ids, -1), 3, align)
    assert torch.equal(fg.lora_f16(x, a, b, route, base=base), base)
    assert not fg.lora_f16(x, a, b, route).any()


def test_no_tokens(fg, dev):
    x, a, b, base, scale, ids = _inputs(4, 3, 64, 136, 16, torch.bfloat16, dev)
    route = fg.route_contiguous(ids[:0], 3, 16)
    assert fg.lora_f16(x[:0], a, b, route, base=base[:0]).shape == (0, 136)


@pytest.mark.parametrize("align,rows", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [3, 700])
def test_rows_of_wider_matrices(fg, dev, monkeypatch, T, dtype, align, rows):
    """x, base and out as columns of wider matrices; what stands beside out is left as it was."""
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    G, K, N, r = 4, 136, 72, 16
    x, a, b, base, scale, ids = _inputs(T, G, K, N, r, dtype, dev)
    route = fg.route_contiguous(ids, G, align)
    want = fg.lora_f16(x, a, b, route, scale=scale, base=base)
    wx = torch.full((T, 3 * K), float("nan"), dtype=dtype, device=dev)
    wx[:, K:2 * K] = x
    wo = torch.full((T, N + 16), 5.0, dtype=dtype, device=dev)
    wo[:, 8:8 + N] = base
    fg.lora_f16(wx[:, K:2 * K], a, b, route, scale=scale, base=wo[:, 8:8 + N], out=wo[:, 8:8 + N])
    assert torch.equal(wo[:, 8:8 + N], want) and (wo[:, :8] == 5.0).all() and (wo[:, 8 + N:] == 5.0).all()
    got = fg.lora_f16(wx[:, K:2 * K], a, b, route, scale=scale, base=base, out=wo[:, 16:16 + N])
    assert torch.equal(got, want)


@pytest.mark.parametrize("align,rows", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
def test_large_and_small_values(fg, dev, monkeypatch, dtype, align, rows):
    """X A^T far above fp16's range beside B far below one, and a token whose own values are tiny:
    the rows of P keep their digits."""
    T, G, K, N, r = 20, 2, 256, 64, 16
    x, a, b, base, scale, ids = _inputs(T, G, K, N, r, dtype, dev, absent=0.0)
    x[::2] *= 64.0
    x[5] *= 2.0 ** -8
    a *= 64.0
    b *= 2.0 ** -9
    scale = scale * 64.0
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    route = fg.route_contiguous(ids, G, align)
    out = fg.lora_f16(x, a, b, route, scale=scale)
    p = torch.einsum("tk,trk->tr", x.double(), a[ids.long()].double()) * scale[ids.long()].double().unsqueeze(1)
    assert p.abs().max() > 70000
    gated_reference.close(out, *ref.lora64(x, a, b, ids, scale, None))


@pytest.mark.parametrize("align,rows", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nans_stay_in_their_tokens(fg, dev, monkeypatch, dtype, align, rows):
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    T, G, K, N, r = 40, 3, 136, 72, 16
    x, a, b, base, scale, ids = _inputs(T, G, K, N, r, dtype, dev, absent=0.0)
    route = fg.route_contiguous(ids, G, align)
    want = fg.lora_f16(x, a, b, route, base=base)
    x2, base2 = x.clone(), base.clone()
    x2[7, 3] = float("nan")
    x2[11, 5] = float("inf")
    base2[13, 2] = float("inf")
    out = fg.lora_f16(x2, a, b, route, base=base2)
    assert torch.isnan(out[7]).all() and not torch.isfinite(out[11]).any() and torch.isinf(out[13, 2])
    keep = torch.ones(T, N, dtype=torch.bool, device=dev)
    keep[[7, 11]] = False
    keep[13, 2] = False
    assert torch.equal(out[keep], want[keep])
    # an adapter that no token has is not looked at
    a[int(ids[0])] = float("nan")
    none = ids != ids[0]
    assert torch.equal(fg.lora_f16(x, a, b, route, base=base)[none], want[none])


def test_bad_rows_are_reported(fg, dev):
    """Rows of another adapter than their block's, adapters and tokens out of range: reported, and
    nothing outside the tensors is touched."""
    T, G, K, N, r = 60, 3, 64, 40, 16
    x, a, b, base, scale, ids = _inputs(T, G, K, N, r, torch.bfloat16, dev, absent=0.0, skew=0.0)
    route = fg.route_contiguous(ids, G, 16)
    want = fg.lora_f16(x, a, b, route, base=base)
    row = int(route.rows[4, 0])
    for field, value in (("m_indices", (int(ids[4]) + 1) % G), ("m_indices", G), ("src", T), ("src", 2 ** 31 - 1)):
        t = getattr(route, field).clone()
        t[row] = value
        if field == "m_indices" and row % 16 == 0:
            continue
        out = base.clone()
        fg.lora_f16(x, a, b, route._replace(**{field: t}), base=out, out=out)
        assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT
        keep = torch.arange(T, device=dev) != 4
        assert torch.equal(out[keep], want[keep])
    m = route.m_indices.clone()
    m[:16] = G + 5                                          # a whole block
    fg.lora_f16(x, a, b, route._replace(m_indices=m), base=base)
    assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT
    assert fg.check_status()[0] == 0


def test_bad_rows_in_wide_blocks_are_reported(fg, dev, monkeypatch):
    """The same where rows come in blocks of 128."""
    monkeypatch.setenv("FGF8_FORCE_TILE", "1x128")
    T, G, K, N, r = 300, 3, 64, 40, 16
    x, a, b, base, scale, ids = _inputs(T, G, K, N, r, torch.bfloat16, dev, absent=0.0, skew=0.0)
    route = fg.route_contiguous(ids, G, 128)
    want = fg.lora_f16(x, a, b, route, base=base)
    other = torch.nonzero(route.m_indices >= 0).view(-1)[5:6]      # a row that is not the first of its block
    token = int(route.src[other])
    for field, value in (("m_indices", (int(ids[token]) + 1) % G), ("m_indices", G), ("src", T), ("src", 2 ** 31 - 1)):
        t = getattr(route, field).clone()
        t[other] = value
        out = base.clone()
        fg.lora_f16(x, a, b, route._replace(**{field: t}), base=out, out=out)
        assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT
        keep = torch.arange(T, device=dev) != token
        assert torch.equal(out[keep], want[keep]) and torch.equal(out[token], base[token])
    m = route.m_indices.clone()
    m[:128] = G + 5                                         # a whole block
    out = base.clone()
    fg.lora_f16(x, a, b, route._replace(m_indices=m), base=out, out=out)
    assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT
    # tiles of 16 that claim to be blocks of 128: rows of other adapters than the first's are left alone
    mixed = fg.route_contiguous(ids, G, 16, M=384)._replace(align=128)
    out = base.clone()
    fg.lora_f16(x, a, b, mixed, base=out, out=out)
    assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT
    first = mixed.m_indices.view(-1, 128)[:, 0].repeat_interleave(128)
    right = torch.zeros(T, dtype=torch.bool, device=dev)
    own = (mixed.src >= 0) & (mixed.m_indices == first)
    right[mixed.src[own].long()] = True
    assert 0 < int(right.sum()) < T and torch.equal(out[right], want[right]) and torch.equal(out[~right], base[~right])
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("align,rows", FORMS)
def test_row_behind_an_empty_first_row_is_reported(fg, dev, monkeypatch, align, rows):
    """A tile or block whose first row has no adapter has none: a row of it that names one is not
    computed, and not passed over in silence."""
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    T, G, K, N, r = 40, 2, 64, 40, 16
    x, a, b, base, scale, ids = _inputs(T, G, K, N, r, torch.bfloat16, dev, absent=0.0, skew=0.0)
    route = fg.route_contiguous(ids, G, align)
    m = route.m_indices.clone()
    m[0] = -1
    out = base.clone()
    fg.lora_f16(x, a, b, route._replace(m_indices=m), base=out, out=out)
    assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT
    held = route.src[:rows][m[:rows] >= 0].long()
    assert held.numel() > 0 and torch.equal(out[held], base[held])
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_wide_blocks_with_few_tokens(fg, dev, monkeypatch, dtype):
    """Blocks of 128 rows of which most are empty, some of them whole blocks, ragged K and N."""
    monkeypatch.setenv("FGF8_FORCE_TILE", "1x128")
    for T, G, K, N, r in [(3, 5, 200, 136, 24), (130, 2, 72, 1000, 128), (257, 40, 328, 72, 56)]:
        x, a, b, base, scale, ids = _inputs(T, G, K, N, r, dtype, dev)
        route = fg.route_contiguous(ids, G, 256)
        out = fg.lora_f16(x, a, b, route, scale=scale, base=base)
        gated_reference.close(out, *ref.lora64(x, a, b, ids, scale, base))
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("align,rows", FORMS)
def test_queue_of_dependent_calls(fg, dev, monkeypatch, align, rows):
    """Calls that each read what the one before wrote, with and without programmatic launches."""
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    T, G, K, r = 260, 3, 256, 32
    x, a, b, _, _, ids = _inputs(T, G, K, K, r, torch.bfloat16, dev)
    before = fg.set_pdl(False)
    try:
        outs = []
        for pdl in (False, True, True):
            fg.set_pdl(pdl)
            y = x.clone()
            for _ in range(40):
                route = fg.route_contiguous(ids, G, align)
                z = fg.lora_f16(y, a, b, route, base=y)
                y = fg.lora_f16(z, a, b, route, base=x)
            outs.append(y)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    finally:
        fg.set_pdl(before)
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("align,rows", FORMS)
def test_streams_and_graphs(fg, dev, monkeypatch, align, rows):
    """On another stream than the current one; captured once and replayed on other inputs, two
    graphs side by side."""
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    T, G, K, N, r = 50, 6, 264, 328, 32
    x, a, b, base, scale, ids = _inputs(T, G, K, N, r, torch.bfloat16, dev)
    route = fg.route_contiguous(ids, G, align)
    want = fg.lora_f16(x, a, b, route, scale=scale, base=base)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream())
    got = fg.lora_f16(x, a, b, route, scale=scale, base=base, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rt = fg.route_contiguous(ids, G, align)
            y = fg.lora_f16(x, a, b, rt, scale=scale, base=base)
            outs.append(fg.lora_f16(x, a, b, rt, scale=scale, base=y, out=y))
        graphs.append(g)
    ids.copy_(ref.random_ids(T, 1, G, 99, 0.2).view(-1))
    x.mul_(0.5)
    streams = [torch.cuda.Stream(dev) for _ in graphs]
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    rt = fg.route_contiguous(ids, G, align)
    y = fg.lora_f16(x, a, b, rt, scale=scale, base=base)
    want = fg.lora_f16(x, a, b, rt, scale=scale, base=y)
    assert all(torch.equal(o, want) for o in outs)
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("T", [1, 40])
def test_beside_a_shared_projection(fg, dev, T):
    """gemm_f16 and lora_f16 on its output, for the layers of a step with one routing; and beside the
    4-bit projection of few tokens."""
    G, K, r = 4, 256, 16
    x, a, b, _, scale, ids = _inputs(T, G, K, K, r, torch.bfloat16, dev)
    w = (torch.randn(K, K, generator=torch.Generator().manual_seed(1)) / K ** 0.5).bfloat16().to(dev)
    route = fg.route_contiguous(ids, G, 16)
    h = x
    for _ in range(3):
        y = fg.gemm_f16(h, w)
        want, bound = ref.lora64(h, a, b, ids, scale, y)
        h = fg.lora_f16(h, a, b, route, scale=scale, base=y, out=y)
        gated_reference.close(h, want, bound)
    if T <= fg.GEMV_MAX_ROWS:
        y = fg.gemv_fp4(x, *fg.quantize_fp4(w, "nv"), "nv")
        want, bound = ref.lora64(x, a, b, ids, scale, y)
        gated_reference.close(fg.lora_f16(x, a, b, route, scale=scale, base=y, out=y), want, bound)
    assert fg.check_status()[0] == 0
