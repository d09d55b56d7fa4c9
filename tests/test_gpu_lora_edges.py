"""GPU tests of lora_f16 at its edges: routings that name rows, adapters and tokens out of range,
infinite values, layouts far larger than their tokens."""
import pytest
import torch

import gated_reference
import routed_reference as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]
# rows of the routing and the form: tiles of 16 in segments of 16 and of 128 rows, blocks of 128
FORMS = [(16, 16), (128, 16), (128, 128)]


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def _inputs(T, G, K, N, r, dtype, dev, seed=0):
    gen = torch.Generator().manual_seed(seed + T + K + N + r)
    x = torch.randn(T, K, generator=gen)
    a, b = torch.randn(G, r, K, generator=gen) / K ** 0.5, torch.randn(G, N, r, generator=gen) / r ** 0.5
    base = torch.randn(T, N, generator=gen)
    ids = ref.random_ids(T, 1, G, seed + T).view(-1)
    return *(t.to(dtype).to(dev) for t in (x, a, b, base)), ids.to(dev)


@pytest.mark.parametrize("align,rows", FORMS)
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_out_of_range_are_reported(fg, dev, monkeypatch, align, rows, in_place):
    """A token whose row is out of range counts as one without an adapter: it gets base, and the call
    reports it, in place too."""
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    T, G, K, N, r = 300, 3, 64, 2056, 16
    x, a, b, base, ids = _inputs(T, G, K, N, r, torch.bfloat16, dev)
    route = fg.route_contiguous(ids, G, align)
    M = route.src.shape[0]
    want = fg.lora_f16(x, a, b, route, base=base)
    assert fg.check_status()[0] == 0
    for t in (4, 31, 299):
        for value in (M, 2 ** 31 - 1, -2, -(2 ** 31)):
            far, src = route.rows.clone(), route.src.clone()
            far[t, 0] = value
            src[route.rows[t, 0].long()] = -1               # nobody's row now
            out = base.clone() if in_place else torch.full_like(base, 3.0)
            fg.lora_f16(x, a, b, route._replace(rows=far, src=src), base=out if in_place else base, out=out)
            assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT, (t, value)
            keep = torch.arange(T, device=dev) != t
            assert torch.equal(out[keep], want[keep]) and torch.equal(out[t], base[t])
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("align,rows", FORMS)
def test_negative_adapters_and_tokens_are_reported(fg, dev, monkeypatch, align, rows):
    """Below -1, which is none, as well as above their range."""
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    T, G, K, N, r = 60, 3, 64, 40, 16
    x, a, b, base, ids = _inputs(T, G, K, N, r, torch.bfloat16, dev)
    route = fg.route_contiguous(ids, G, align)
    want = fg.lora_f16(x, a, b, route, base=base)
    at = int(torch.nonzero(route.m_indices >= 0)[5])        # not the first of its tile or block
    token = int(route.src[at])
    for field in ("m_indices", "src"):
        for value in (-2, -(2 ** 31)):
            t = getattr(route, field).clone()
            t[at] = value
            out = base.clone()
            fg.lora_f16(x, a, b, route._replace(**{field: t}), base=out, out=out)
            assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT, (field, value)
            keep = torch.arange(T, device=dev) != token
            assert torch.equal(out[keep], want[keep]) and torch.equal(out[token], base[token])
    m = route.m_indices.clone()
    m[0] = -2                                               # the first of its tile: the tile has no adapter
    out = base.clone()
    fg.lora_f16(x, a, b, route._replace(m_indices=m), base=out, out=out)
    assert fg.check_status()[0] == fg.ERR_DEVICE_INPUT
    assert fg.check_status()[0] == 0


# ----------------------------------------------------------------- infinities
def _lora_ieee(x, a, b, ids, scale, base):
    """The definition term by term in 64 bits, infinities and NaN as IEEE arithmetic has them."""
    x, a, b, base, ids = x.double().cpu(), a.double().cpu(), b.double().cpu(), base.double().cpu(), ids.long().cpu()
    p = (x.unsqueeze(1) * a[ids]).sum(-1)
    if scale is not None:
        p = p * scale.double().cpu()[ids].unsqueeze(1)
    return base + (p.unsqueeze(1) * b[ids]).sum(-1)


def _same_kinds(out, want, bound_of):
    """NaN and infinities where the definition has them, the rest within its bound."""
    got = out.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"NaN: {int(torch.isnan(got).sum())}, the definition {int(torch.isnan(want).sum())}"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    fine = torch.isfinite(want)
    value, bound = (t.cpu()[fine] for t in bound_of)
    assert ((got[fine] - value).abs() <= bound).all()


# ranks that are not their padded size: columns of P from r on do not exist
@pytest.mark.parametrize("align,rows", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("r", [8, 16, 24, 40, 72])
def test_infinite_x_or_scale(fg, dev, monkeypatch, r, dtype, align, rows):
    """A token with an infinity, and an adapter with an infinite scale, give the infinities of the
    definition: every term of a column has one sign."""
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    T, G, K, N = 24, 2, 136, 72
    x, a, b, base, ids = _inputs(T, G, K, N, r, dtype, dev)
    route = fg.route_contiguous(ids, G, align)
    t = 11
    g = int(ids[t])
    scale = torch.tensor([0.75, 0.75], device=dev)
    columns = torch.where(torch.arange(N, device=dev) % 3 == 0, -1.0, 1.0).to(dtype)
    b[g] = (b[g].abs() + 2.0 ** -10) * torch.sign(a[g, :, 5]) * columns.unsqueeze(1)
    a[g, :, 5] += torch.sign(a[g, :, 5]) * 2.0 ** -10
    bounds = ref.lora64(x, a, b, ids, scale, base)          # of the tokens that stay finite
    far = x.clone()
    far[t, 5] = float("inf")
    want = _lora_ieee(far, a, b, ids, scale, base)
    assert torch.isinf(want[t]).all() and torch.isfinite(want[torch.arange(T) != t]).all()
    _same_kinds(fg.lora_f16(far, a, b, route, scale=scale, base=base), want, bounds)
    # P of one sign per rank row: all tokens of the adapter see sgn(A) K times
    x[ids == g] = x[ids == g].abs() + 0.5
    a[g] = a[g].abs() + 2.0 ** -10
    b[g] = (b[g].abs() + 2.0 ** -10) * columns.unsqueeze(1)
    scale[g] = float("inf")
    want = _lora_ieee(x, a, b, ids, scale, base)
    mine = (ids == g).cpu()
    assert torch.isinf(want[mine]).all() and torch.isfinite(want[~mine]).all()
    bounds = ref.lora64(x, a, b, torch.where(ids == g, -1, ids), torch.ones_like(scale) * 0.75, base)
    _same_kinds(fg.lora_f16(x, a, b, route, scale=scale, base=base), want, bounds)
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("align,rows", FORMS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("r", [8, 24, 64, 128])
def test_infinite_weights(fg, dev, monkeypatch, r, dtype, align, rows):
    """Infinities in B meet each element of P once, whatever parts P is kept in: an exact one has no
    rest, others have one of the other sign.  An infinity in A makes one element of a row of P
    infinite and leaves its others what they are."""
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
    T, G, K, N = 40, 2, 136, 136
    x, a, b, base, ids = _inputs(T, G, K, N, r, dtype, dev)
    ids[:20], ids[20:] = 0, 1
    route = fg.route_contiguous(ids, G, align)
    # exact P, among them zeros: tokens 0 .. 3 are one column of A times small whole numbers
    x[:4] = 0.0
    x[:4, 0] = torch.tensor([1.0, -2.0, 3.0, 0.0]).to(dtype).to(dev)
    bounds = ref.lora64(x, a, b, ids, None, base)
    far = b.clone()
    far[0, 7, 3], far[0, 100, 0], far[1, 64, r - 1] = float("inf"), float("-inf"), float("inf")
    want = _lora_ieee(x, a, far, ids, None, base)
    assert int(torch.isinf(want).sum()) == 20 + 2 * 19 and torch.isnan(want[3, 7]) and torch.isnan(want[3, 100])
    _same_kinds(fg.lora_f16(x, a, far, route, base=base), want, bounds)
    # one infinite element of P beside large ones of the other sign
    wide = a.clone()
    wide[1] *= -1024.0
    wide[1, 2, 9] = float("inf")
    x[20:] = x[20:].abs() * 1024.0 + 1.0
    b[1] = b[1].abs() + 2.0 ** -10
    want = _lora_ieee(x, wide, b, ids, None, base)
    assert torch.isinf(want[20:]).all() and torch.isfinite(want[:20]).all()
    _same_kinds(fg.lora_f16(x, wide, b, route, base=base), want, bounds)
    assert fg.check_status()[0] == 0


def test_infinite_weights_in_place_and_without_a_base(fg, dev, monkeypatch):
    T, G, K, N, r = 200, 3, 264, 200, 32
    for dtype in TYPES:
        x, a, b, base, ids = _inputs(T, G, K, N, r, dtype, dev)
        b[1, 13, 4] = float("inf")
        b[2, 190, 31] = float("nan")
        zero = torch.zeros_like(base)
        for align, rows in FORMS:
            monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{rows}")
            route = fg.route_contiguous(ids, G, align)
            finite = torch.nan_to_num(b, nan=0.0, posinf=0.0)
            out = base.clone()
            fg.lora_f16(x, a, b, route, base=out, out=out)
            _same_kinds(out, _lora_ieee(x, a, b, ids, None, base), ref.lora64(x, a, finite, ids, None, base))
            _same_kinds(fg.lora_f16(x, a, b, route), _lora_ieee(x, a, b, ids, None, zero), ref.lora64(x, a, finite, ids, None, zero))
    assert fg.check_status()[0] == 0


# ----------------------------------------------------------------- large layouts
def test_a_layout_far_larger_than_its_tokens(fg, dev, monkeypatch):
    """2^28 rows for two tokens: 2^24 tiles, whose warps would not be counted in 32 bits if each tile
    had the 32 CTAs of a call with two."""
    monkeypatch.setenv("FGF8_FORCE_TILE", "1x16")
    T, G, K, N, r = 2, 1, 2048, 8192, 16
    x, a, b, base, ids = _inputs(T, G, K, N, r, torch.bfloat16, dev)
    ids[1] = -1
    route = fg.route_contiguous(ids, G, 16, M=1 << 28)
    out = fg.lora_f16(x, a, b, route, base=base, out=torch.full_like(base, 3.0))
    gated_reference.close(out, *ref.lora64(x, a, b, ids, None, base))
    assert torch.equal(out[1], base[1])
    assert fg.check_status()[0] == 0
