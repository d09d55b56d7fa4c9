"""GPU tests of lora_f16 at its edges: routings that name rows, adapters and tokens out of range."""
import pytest
import torch

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
