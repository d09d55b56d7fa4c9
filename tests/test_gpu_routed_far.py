"""GPU tests of the routed operators where offsets pass 2^32 bytes, and of calls of several
threads at once."""
import threading

import pytest
import torch

import gated_reference
import routed_reference as ref

pytestmark = pytest.mark.gpu
T, G, H, K = 70000, 3, 16384, 2                            # 140000 rows of 16384: 2.3e9 elements


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def _noise(rows, cols, dev, seed):
    gen = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(rows, cols, generator=gen, device=dev, dtype=torch.bfloat16)


def _far(fg, dev):
    """A routing, and tokens with rows at the far end of the layout."""
    r = fg.route_contiguous(ref.random_ids(T, K, G, 5, 0.001).to(dev), G)
    last = r.rows.amax(1).topk(40).indices
    tokens = torch.unique(torch.cat((last, torch.arange(T - 40, T, device=dev), torch.arange(8, device=dev))))
    assert int(r.rows[tokens].max()) * H > 2 ** 31
    return r, tokens


def test_dispatch_far(fg, dev):
    r, tokens = _far(fg, dev)
    x = _noise(T, H, dev, 1)
    xs = fg.dispatch_f16(x, r)
    codes, table = fg.dispatch_fp8(x, r, 1)
    want_codes, want_table = fg.quantize_1x128(x[tokens].contiguous(), 1)
    for j in range(K):
        has = r.rows[tokens, j] >= 0
        at = r.rows[tokens, j][has].long()
        assert torch.equal(xs[at], x[tokens[has]])
        assert torch.equal(codes[at], want_codes[has])
        assert torch.equal(table[:, at], want_table[:, :len(tokens)][:, has])
    empty = torch.nonzero(r.src < 0).view(-1)
    assert len(empty) > 0 and not xs[empty].any()
    assert fg.check_status()[0] == 0


def test_combine_far(fg, dev):
    r, tokens = _far(fg, dev)
    M = r.src.shape[0]
    ys, dy = _noise(M, H, dev, 2), _noise(T, H, dev, 3)
    w = torch.randn(T, K, generator=torch.Generator().manual_seed(4)).to(dev)
    y = fg.combine_f16(ys, w, r)
    gated_reference.close(y[tokens], *ref.combine64(ys, w[tokens], r.rows[tokens], ys.dtype))
    del y
    dys, dw = fg.combine_f16_backward(dy, ys, w, r)
    # the same tokens in a layout of their own
    rows = r.rows[tokens]
    has = rows >= 0
    near = torch.where(has, has.view(-1).cumsum(0).view(rows.shape) - 1, -1).int()
    n = int(has.sum())
    (want, want_dw), (bound, bound_dw) = ref.combine_backward64(dy[tokens], ys[rows[has].long()], w[tokens], near, n, ys.dtype)
    gated_reference.close(dys[rows[has].long()], want, bound)
    gated_reference.close(dw[tokens], want_dw, bound_dw)
    assert not dys[torch.nonzero(r.src < 0).view(-1)].any()
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("align", [16, 128])
def test_lora_far(fg, dev, monkeypatch, align):
    """Rows of x, base and out 32768 elements apart."""
    monkeypatch.setenv("FGF8_FORCE_TILE", f"1x{align}")
    N, k, r = 32768, 72, 8
    wide = _noise(T, N, dev, 6)
    x = wide[:, N - k:]
    a, b = _noise(G, r * k, dev, 7).view(G, r, k), _noise(G, N * r, dev, 8).view(G, N, r)
    scale = torch.tensor([0.5, -1.0, 2.0], device=dev)
    ids = ref.random_ids(T, 1, G, 9, 0.01).view(-1).to(dev)
    route = fg.route_contiguous(ids, G, align)
    out = fg.lora_f16(x, a, b, route, scale=scale, base=wide)
    assert fg.last_tile().endswith(f"x{align}")
    absent = torch.nonzero(ids < 0).view(-1)[-4:]
    tokens = torch.cat((torch.arange(4, device=dev), torch.arange(T - 24, T, device=dev), absent))
    gated_reference.close(out[tokens], *ref.lora64(x[tokens], a, b, ids[tokens], scale, wide[tokens]))
    assert torch.equal(out[absent], wide[absent])
    assert fg.check_status()[0] == 0


def test_threads_on_streams(fg, dev):
    """Several threads, each on a stream of its own, the same results as one after the other."""
    H, r = 1024, 16

    def work(seed):
        t = 300 + 50 * seed
        x = _noise(t, H, dev, seed)
        ids = ref.random_ids(t, 3, 5, seed, 0.1).to(dev)
        w = torch.rand(t, 3, generator=torch.Generator().manual_seed(seed)).to(dev)
        a, b = _noise(5, r * H, dev, seed + 20).view(5, r, H), _noise(5, H * r, dev, seed + 30).view(5, H, r)
        torch.cuda.current_stream().synchronize()
        out = []
        for _ in range(20):
            route = fg.route_contiguous(ids, 5, 16)
            xs = fg.dispatch_f16(x, route)
            y = fg.combine_f16(xs, w, route)
            dys, dw = fg.combine_f16_backward(y, xs, w, route)
            one = fg.route_contiguous(ids[:, 0].contiguous(), 5, 128)
            out = [route.rows, route.src, xs, y, dys, dw, fg.lora_f16(y, a, b, one, base=x)]
        return out

    want = [work(s) for s in range(4)]
    torch.cuda.synchronize()
    got = [None] * 4

    def run(s):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[s] = work(s)

    threads = [threading.Thread(target=run, args=(s,)) for s in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert g is not None and all(torch.equal(p, q) for p, q in zip(g, w))
    assert fg.check_status()[0] == 0
