"""CPU checks of the routing, dispatch, combine and adapter operators' refusals: the C ABI
rejects invalid calls on the host, the binding rejects tensors of another size, type or
layout.  Nothing reaches a GPU."""
import ctypes

import pytest
import torch

import routed_reference as ref

P, I, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
AL, MIS = P(0x10000), P(0x10008)     # never dereferenced: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    from fine_grained_fp8_persistent_gb300 import build
    lib = ctypes.CDLL(build.build())
    lib.fgf8_last_error.restype = ctypes.c_char_p
    lib.fgf8_route_rows.restype = LL
    return lib


def _err(lib):
    return lib.fgf8_last_error().decode()


def _fn(lib, name, pointers, ints, longs=0):
    f = getattr(lib, name)
    f.argtypes = [P] * pointers + [I] * ints + [LL] * longs + ([I] if longs else []) + [P]
    return f


def test_route_refusals(lib):
    f = _fn(lib, "route_contiguous", 6, 6)
    ok = [AL] * 6
    assert f(*ok, -1, 2, 4, 128, 512, 0, None) == 1
    assert f(*ok, 4, 0, 4, 128, 512, 0, None) == 1
    assert f(*ok, 4, 2, 0, 128, 512, 0, None) == 1
    assert f(*ok, 4, 2, 1025, 128, 1 << 20, 0, None) == 2 and "1024" in _err(lib)
    assert f(*ok, 4, 2, 4, 0, 512, 0, None) == 1
    assert f(*ok, 4, 2, 4, 128, 500, 0, None) == 1 and "segments" in _err(lib)
    assert f(*ok, 4, 2, 4, 128, 384, 0, None) == 1 and "512" in _err(lib)      # 4 groups may have entries
    assert f(*ok, 1 << 30, 2, 4, 1, 1 << 30, 0, None) == 2                      # 2^31 entries
    assert f(None, *ok[1:], 4, 2, 4, 128, 512, 0, None) == 1
    assert f(MIS, *ok[1:], 4, 2, 4, 128, 512, 0, None) == 3
    assert f(*ok[:3], None, *ok[4:], 4, 2, 4, 128, 512, 1, None) == 1
    m = _fn(lib, "route_masked", 4, 5)
    ok = [AL] * 4
    assert m(*ok, 4, 2, 4, 0, 0, None) == 1
    assert m(*ok, 4, 2, 0, 8, 0, None) == 1
    assert m(*ok, 4, 2, 1000, 1 << 22, 0, None) == 2 and "rows above" in _err(lib)
    assert m(*ok[:2], None, AL, 4, 2, 4, 8, 0, None) == 1
    assert m(AL, MIS, AL, AL, 4, 2, 4, 8, 0, None) == 3


def test_route_rows_hold_any_split(lib):
    rows = lib.fgf8_route_rows
    assert rows(0, 8, 32, 128) == 0 and rows(1, 1, 32, 128) == 128 and rows(1, 8, 32, 128) == 1024
    assert rows(8192, 8, 32, 128) == 65536 + 31 * 128
    assert rows(-1, 1, 1, 1) == rows(1, 0, 1, 1) == rows(1, 1, 0, 1) == rows(1, 1, 1, 0) == -1
    assert rows(1 << 30, 1, 1024, 128) > 1 << 30
    for T, k, G, align in [(1, 1, 1, 16), (7, 3, 5, 16), (40, 2, 9, 128), (33, 1, 64, 1), (50, 4, 3, 7)]:
        most = 0
        for seed in range(30):
            ids = ref.random_ids(T, k, G, seed, skew=seed / 30)
            most = max(most, int(ref.route(ids.numpy(), G, align)[4][-1]))
        # one entry in each group and the rest in one is the split that needs most
        flat = (list(range(min(G, T * k))) + [0] * (T * k))[: T * k]
        worst = int(ref.route(torch.tensor(flat).view(T, k).numpy(), G, align)[4][-1])
        bound = rows(T, k, G, align)
        assert max(most, worst) <= bound and bound % align == 0


def test_dispatch_refusals(lib):
    f = _fn(lib, "dispatch_f16", 4, 4)
    ok = [AL] * 4
    assert f(*ok, -1, 2, 64, 128, None) == 1
    assert f(*ok, 4, 2, 0, 128, None) == 1
    assert f(*ok, 4, 2, 64, -1, None) == 1
    assert f(*ok, 4, 2, 60, 128, None) == 2 and "multiple of 8" in _err(lib)
    assert f(AL, None, AL, AL, 4, 2, 64, 128, None) == 1
    assert f(AL, AL, AL, MIS, 4, 2, 64, 128, None) == 3
    assert f(None, None, None, None, 0, 2, 64, 0, None) == 0
    q = _fn(lib, "dispatch_fp8", 4, 6)
    assert q(*ok, 4, 2, 64, 128, 0, 0, None) == 2 and "multiple of 128" in _err(lib)
    assert q(*ok, 4, 2, 128, 128, 0, 2, None) == 1 and "format" in _err(lib)
    assert q(*ok, 4, 2, 128, 100, 30, 0, None) == 1 and "slots" in _err(lib)
    assert q(*ok, 4, 2, 128, 100, -1, 0, None) == 1
    assert q(AL, AL, MIS, AL, 4, 2, 128, 128, 0, 0, None) == 3
    assert q(None, None, None, None, 0, 2, 128, 128, 0, 0, None) == 0


def test_combine_refusals(lib):
    f = _fn(lib, "combine_f16", 4, 5)
    ok = [AL] * 4
    assert f(*ok, 4, 2, 64, 128, 2, None) == 1 and "dtype" in _err(lib)
    assert f(*ok, 4, 2, 12, 128, 0, None) == 2
    assert f(*ok, 4, -2, 64, 128, 0, None) == 1
    assert f(AL, MIS, AL, AL, 4, 2, 64, 128, 0, None) == 3
    assert f(None, AL, AL, AL, 4, 2, 64, 128, 0, None) == 1
    assert f(None, None, None, None, 0, 2, 64, 128, 0, None) == 0
    d = _fn(lib, "dispatch_f16_backward", 3, 5)
    assert d(AL, AL, AL, 4, 2, 20, 128, 0, None) == 2 and "dispatch_f16_backward" in _err(lib)
    assert d(AL, None, AL, 4, 2, 64, 128, 0, None) == 1
    b = _fn(lib, "combine_f16_backward", 7, 5)
    ok = [AL] * 7
    assert b(*ok, 4, 2, 64, 128, -1, None) == 1
    assert b(*ok, 4, 2, 65, 128, 0, None) == 2
    assert b(AL, AL, None, *ok[3:], 4, 2, 64, 128, 0, None) == 1
    assert b(*ok[:6], MIS, 4, 2, 64, 128, 0, None) == 3
    assert b(*[None] * 7, 0, 2, 64, 0, 0, None) == 0


def test_lora_refusals(lib):
    f = _fn(lib, "lora_f16", 9, 7, 3)
    ok = [AL] * 4 + [AL] * 5

    def call(T=4, K=64, N=32, r=16, G=2, M=32, align=16, ldx=64, ldb=32, ldo=32, dtype=0, ptrs=ok):
        return f(*ptrs, T, K, N, r, G, M, align, ldx, ldb, ldo, dtype, None)
    assert call(T=-1) == 1 and call(r=0) == 1 and call(G=0) == 1 and call(M=-16) == 1
    assert call(K=60, ldx=64) == 2 and call(N=20) == 2
    assert call(r=12) == 2 and "rank 12" in _err(lib)
    assert call(r=136) == 2
    assert call(align=8) == 2 and "align=8" in _err(lib)
    assert call(M=40) == 1 and call(M=64, align=128) == 1 and call(align=0) == 2
    assert call(dtype=2) == 1
    assert call(ldx=56) == 1 and "apart" in _err(lib)
    assert call(ldo=24) == 1 and call(ldb=24) == 1
    assert call(ldx=68) == 3 and call(ldo=36, ldb=36) == 3
    assert call(ldb=40) == 1 and "base is out" in _err(lib)                     # the same pointer
    assert call(ptrs=[AL, None] + ok[2:]) == 1
    assert call(ptrs=ok[:3] + [MIS] + ok[4:]) == 3                              # scale
    assert call(ptrs=[None] * 9, T=0) == 0


def test_lora_without_rows(lib):
    """Tokens need rows, even when none has an adapter and out is another matrix than base."""
    f = _fn(lib, "lora_f16", 9, 7, 3)
    for out, ldo in ((AL, 32), (P(0x20000), 40)):
        assert f(*[AL] * 8, out, 4, 64, 32, 16, 2, 0, 16, 64, 32, ldo, 0, None) == 1 and "no rows" in _err(lib)
    assert f(*[AL] * 9, 0, 64, 32, 16, 2, 0, 16, 64, 32, 32, 0, None) == 0


# ----------------------------------------------------------------- the binding
@pytest.fixture()
def fg(monkeypatch):
    from fine_grained_fp8_persistent_gb300 import binding
    calls = []
    monkeypatch.setattr(binding, "_launch", lambda name, stream, tensors, ints, strided=(): calls.append((name, tensors, ints)))
    binding.calls = calls
    return binding


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _refused(bad):
    for call, match in bad:
        with pytest.raises(ValueError, match=match):
            call()


def test_binding_route(fg):
    ids = z(5, 3, dtype=torch.int32)
    r = fg.route_contiguous(ids, 4)
    assert r.rows.shape == (5, 3) and r.src.shape == r.m_indices.shape == (512,) and r.counts.shape == (4,) and r.starts.shape == (5,)
    assert (r.align, r.slots) == (128, 0) and fg.calls[-1][2] == (5, 3, 4, 128, 512, 0)
    r = fg.route_contiguous(z(5, dtype=torch.int64), 4, align=16, M=128)
    assert r.rows.shape == (5, 1) and r.src.shape == (128,) and fg.calls[-1][2] == (5, 1, 4, 16, 128, 1)
    r = fg.route_masked(ids, 4, 7)
    assert r.src.shape == (28,) and r.m_indices is None and r.starts is None and r.slots == 7
    _refused([(lambda: fg.route_contiguous(ids.float(), 4), "int32 or int64"), (lambda: fg.route_masked(z(2, 2, 2, dtype=torch.int32), 4, 7), "ids")])


def test_binding_dispatch_and_combine(fg):
    ids, x = z(5, 3, dtype=torch.int32), z(5, 256)
    r, m = fg.route_contiguous(ids, 4), fg.route_masked(ids, 4, 7)
    assert fg.dispatch_f16(x, r).shape == (512, 256)
    assert fg.calls[-1][1][2] is r.src                                          # empty rows become zeros
    fg.dispatch_f16(x, m)
    assert fg.calls[-1][1][2] is None                                           # here they stay
    xq, sfa = fg.dispatch_fp8(x, r, "f32")
    assert xq.shape == (512, 256) and sfa.shape == (2, 512) and sfa.dtype == torch.float32
    xq, sfa = fg.dispatch_fp8(x, m, "ue8m0")
    assert xq.shape == (4, 7, 256) and sfa.shape == (4, 1, 8) and sfa.dtype == torch.int32
    w = z(5, 3, dtype=torch.float32)
    ys = z(512, 64)
    y = fg.combine_f16(ys, w, r)
    assert y.shape == (5, 64) and fg.combine_f16(z(4, 7, 64), None, m).shape == (5, 64)
    dys, dw = fg.combine_f16_backward(y, ys, w, r)
    assert dys.shape == ys.shape and dw.shape == w.shape and fg.dispatch_f16_backward(z(512, 256), r).shape == x.shape
    n = len(fg.calls)
    _refused([
        (lambda: fg.dispatch_f16(x[:4], r), "rows"),
        (lambda: fg.dispatch_f16(x.float(), r), "fp16 or bf16"),
        (lambda: fg.dispatch_f16(x, r, out=z(512, 128)), "out"),
        (lambda: fg.dispatch_f16(x, r, out=z(512, 256).half()), "out"),
        (lambda: fg.dispatch_f16(x, r._replace(src=r.src.long())), "src"),
        (lambda: fg.dispatch_fp8(x.half(), r, 0), "bf16"),
        (lambda: fg.dispatch_fp8(x, r, 0, xq=z(511, 256, dtype=torch.uint8)), "xq"),
        (lambda: fg.dispatch_fp8(x, r, 0, sfa=z(2, 508, dtype=torch.float32)), "sfa"),
        (lambda: fg.combine_f16(z(511, 64), w, r), "ys"),
        (lambda: fg.combine_f16(ys, w.half(), r), "w"),
        (lambda: fg.combine_f16(ys, w[:, :2], r), "w"),
        (lambda: fg.combine_f16(ys, w, r, out=z(4, 64)), "out"),
        (lambda: fg.combine_f16_backward(y.half(), ys, w, r), "ys"),
        (lambda: fg.combine_f16_backward(y, z(512, 72), w, r), "ys"),
        (lambda: fg.combine_f16_backward(y, ys, w, r, dw=z(5, 3)), "dw"),
        (lambda: fg.combine_f16_backward(y, ys, w, r, dys=z(512, 72)), "dys"),
        (lambda: fg.dispatch_f16_backward(z(100, 256), r), "dxs"),
    ])
    assert len(fg.calls) == n


def test_binding_lora(fg):
    T, K, N, G, rank = 5, 64, 32, 3, 16
    x, a, b = z(T, K), z(G, rank, K), z(G, N, rank)
    r = fg.route_contiguous(z(T, dtype=torch.int32), G, align=16)
    assert fg.lora_f16(x, a, b, r).shape == (T, N)
    assert fg.calls[-1][2] == (T, K, N, rank, G, 48, 16, 64, 0, 32, 1)
    wide = z(T, 3 * N)
    out = wide[:, N:2 * N]
    assert fg.lora_f16(x, a, b, r, base=out, out=out) is out
    assert fg.calls[-1][2][-4:] == (64, 96, 96, 1)
    _refused([
        (lambda: fg.lora_f16(x.float(), a, b, r), "fp16 or bf16"),
        (lambda: fg.lora_f16(x, a.half(), b, r), "a"),
        (lambda: fg.lora_f16(x, a[0], b, r), "a and b"),
        (lambda: fg.lora_f16(x, a, b[:2], r), "b"),
        (lambda: fg.lora_f16(x, a, z(G, N, 8), r), "b"),
        (lambda: fg.lora_f16(x[:4], a, b, r), "route.rows"),
        (lambda: fg.lora_f16(x, a, b, fg.route_contiguous(z(T, 2, dtype=torch.int32), G, align=16)), "route"),
        (lambda: fg.lora_f16(x, a, b, fg.route_masked(z(T, dtype=torch.int32), G, 16)), "route"),
        (lambda: fg.lora_f16(x, a, b, fg.route_contiguous(z(T, dtype=torch.int32), G, align=8)), "align 8"),
        (lambda: fg.lora_f16(x, a, b, r, scale=z(G)), "scale"),
        (lambda: fg.lora_f16(x, a, b, r, base=z(T, K)), "base"),
        (lambda: fg.lora_f16(x, a, b, r, out=z(T, N).half()), "out"),
        (lambda: fg.lora_f16(x.t().contiguous().t(), a, b, r), "strides"),
        (lambda: fg.lora_f16(x, a, b, r, out=z(N).expand(T, N)), "strides"),
    ])


def test_strided_tensors_pass_the_launch_only_where_named():
    from fine_grained_fp8_persistent_gb300 import binding

    class Fake:
        is_cuda = True

        def is_contiguous(self):
            return False

        def get_device(self):
            return 0

        def data_ptr(self):
            return 0x10000
    with pytest.raises(ValueError, match="contiguous"):
        binding._launch("lora_f16", None, (Fake(), Fake()), (), strided=(0,))


def test_package_exports():
    import fine_grained_fp8_persistent_gb300 as pkg
    for name in ("Route", "route_contiguous", "route_masked", "route_rows", "dispatch_f16", "dispatch_fp8", "dispatch_f16_backward",
                 "combine_f16", "combine_f16_backward", "lora_f16"):
        assert callable(getattr(pkg, name))
    assert pkg.route_rows(8192, 8, 32) == 65536 + 31 * 128
