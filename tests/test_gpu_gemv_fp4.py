"""GPU tests of gemv_fp4 and gated_gemv_fp4 against their definition in 64 bits, on
weights in the oracle's 4-bit layouts."""
import numpy as np
import pytest
import torch

import gated_reference as ref

pytestmark = pytest.mark.gpu
FMTS = [0, 1]          # MXFP4, NVFP4
TYPES = [torch.bfloat16, torch.float16]
SHAPES = [(1, 1, 64), (1, 16, 128), (1, 100, 448), (1, 257, 7168), (1, 2048, 1024), (2, 3, 192), (3, 15, 320), (4, 33, 64), (5, 48, 640),
          (7, 17, 256), (8, 64, 512), (8, 300, 2112), (9, 31, 128), (12, 129, 960), (15, 50, 4096), (16, 16, 64),
          (16, 1000, 7168), (1, 40, 16448), (16, 24, 16448)]


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def _weights(oracle, N, K, fmt, seed, dev):
    gen = np.random.default_rng(seed)
    w = gen.standard_normal((N, K)).astype(np.float32) / np.sqrt(K)
    w *= np.exp2(gen.integers(-3, 4, (N, 1))).astype(np.float32)
    q, sf = oracle.quantize_fp4(w, fmt)
    w64 = torch.from_numpy(oracle.dequantize_fp4(q, sf, fmt))
    return torch.from_numpy(q).to(dev), torch.from_numpy(sf).to(dev), w64


def _x(M, K, dtype, seed, dev):
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(seed))
    x[:, :: max(1, K // 5)] *= 30.0
    return x.to(dtype).to(dev)


def _check(got, x, w64, what=""):
    R, T = ref.unit(x.dtype)
    y, err = ref.gemv64(x, w64)
    ref.close(got, y, err + R * (y.abs() + err) + T, what)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemv(fg, dev, oracle, M, N, K, dtype, fmt):
    wq, sf, w64 = _weights(oracle, N, K, fmt, N + K, dev)
    x = _x(M, K, dtype, M + K, dev)
    y = fg.gemv_fp4(x, wq, sf, fmt)
    _check(y, x, w64)
    assert torch.equal(y, fg.gemv_fp4(x, wq, sf, fmt))


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES[:-2:2] + SHAPES[-2:])
def test_gated_gemv(fg, dev, oracle, M, N, K, dtype, fmt, act):
    gq, gs, g64 = _weights(oracle, N, K, fmt, N + K, dev)
    uq, us, u64 = _weights(oracle, N, K, fmt, N + K + 1, dev)
    x = _x(M, K, dtype, M + K, dev)
    h = fg.gated_gemv_fp4(x, gq, gs, uq, us, fmt, act)
    g, dg = ref.gemv64(x, g64)
    u, du = ref.gemv64(x, u64)
    want, bound = ref.gate64(g, dg, u, du, act, dtype)
    ref.close(h, want, bound)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 8, 16])
def test_every_code_and_scale(fg, dev, oracle, fmt, M):
    """Every 4-bit code under every finite scale byte (MXFP4: 2^-127 .. 2^127, NVFP4: all
    E4M3 values, negative ones and zero too), one scale per weight row, alternating over
    the row's groups with the neutral one.  A single non-zero x keeps each product apart."""
    sv = 32 if fmt == 0 else 16
    scales = np.arange(0, 255) if fmt == 0 else np.array([b for b in range(256) if b & 0x7F != 0x7F])
    N, K = len(scales), 128
    codes = np.tile(np.arange(16, dtype=np.uint8), (N, K // 16))
    q = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    shape, _ = oracle.fp4_sf_shape(N, K, fmt)
    b = np.zeros((shape[0], shape[1], 4), np.uint8)
    for grp in range(K // sv):
        b[grp // 4, :N, grp % 4] = scales if grp % 2 else (127 if fmt == 0 else 0x38)
    sf = b.view(np.int32).reshape(shape)
    w64 = torch.from_numpy(oracle.dequantize_fp4(q, sf, fmt))
    wq, sfd = torch.from_numpy(q).to(dev), torch.from_numpy(sf.copy()).to(dev)
    for k in (5, sv + 1, sv + 2, sv + 7, sv + 15, K - 1, K - 8):
        x = torch.zeros(M, K, dtype=torch.bfloat16, device=dev)
        x[:, k] = 0.03125
        _check(fg.gemv_fp4(x, wq, sfd, fmt), x, w64, f"k = {k}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [2, 9])
def test_nan_scales_stay_in_their_rows(fg, dev, oracle, fmt, M):
    """A NaN scale (E8M0 byte 255, E4M3 0x7F) makes its own weight row's outputs NaN, no others."""
    N, K = 37, 512
    wq, sf, w64 = _weights(oracle, N, K, fmt, 12, dev)
    x = _x(M, K, torch.bfloat16, 13, dev)
    clean = fg.gemv_fp4(x, wq, sf, fmt)
    b = sf.cpu().numpy().view(np.uint8).reshape(*sf.shape, 4).copy()
    b[1, 20, 2] = 255 if fmt == 0 else 0x7F
    bad = torch.from_numpy(b.view(np.int32).reshape(tuple(sf.shape))).to(dev)
    y = fg.gemv_fp4(x, wq, bad, fmt)
    rows = torch.arange(N, device=dev) != 20
    assert torch.isnan(y[:, 20]).all() and torch.equal(y[:, rows], clean[:, rows])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [2, 13])
def test_many_rows(fg, dev, oracle, fmt, M):
    """More weight rows than one round of tiles holds, plain and gated."""
    N, K = 45001, 192
    wq, sf, w64 = _weights(oracle, N, K, fmt, 14, dev)
    x = _x(M, K, torch.float16, 15, dev)
    y = fg.gemv_fp4(x, wq, sf, fmt)
    _check(y, x, w64)
    h = fg.gated_gemv_fp4(x, wq, sf, wq, sf, fmt)
    g, dg = ref.gemv64(x, w64)
    ref.close(h, *ref.gate64(g, dg, g, dg, "silu", x.dtype))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(8, 512, 4096), (8, 2048, 7168), (16, 4096, 4096), (7, 333, 7232), (16, 2048, 16384)])
def test_split_reductions(fg, dev, oracle, M, N, K, dtype, fmt):
    """Sizes whose reduction a cluster of 2, 4 or 8 CTAs shares, one with an odd last share."""
    wq, sf, w64 = _weights(oracle, N, K, fmt, 21, dev)
    x = _x(M, K, dtype, 22, dev)
    y = fg.gemv_fp4(x, wq, sf, fmt)
    _check(y, x, w64)
    assert torch.equal(y, fg.gemv_fp4(x, wq, sf, fmt))


@pytest.mark.parametrize("fmt", FMTS)
def test_wide_range_of_x(fg, dev, oracle, fmt):
    """Rows of X that span 2^-100 .. 2^100, one row each, and rows that mix sizes 2^30 apart."""
    M, N, K = 8, 40, 256
    wq, sf, w64 = _weights(oracle, N, K, fmt, 3, dev)
    x = _x(M, K, torch.bfloat16, 4, dev).float()
    x *= torch.tensor([1e-30, 1e-10, 1e-3, 1.0, 1e3, 1e10, 1e20, 1e30], device=dev)[:, None]
    x = x.to(torch.bfloat16)
    _check(fg.gemv_fp4(x, wq, sf, fmt), x, w64)
    x[:, ::2] = x[:, ::2] * 2.0 ** -30
    _check(fg.gemv_fp4(x, wq, sf, fmt), x, w64)
    x[:, 1::2] = 0.0                                     # only the small ones are left
    _check(fg.gemv_fp4(x, wq, sf, fmt), x, w64)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 3, 16])
def test_non_finite_rows_stay_to_themselves(fg, dev, oracle, fmt, dtype, M):
    N, K = 50, 320
    wq, sf, w64 = _weights(oracle, N, K, fmt, 6, dev)
    x = _x(M, K, dtype, 7, dev)
    clean = fg.gemv_fp4(x, wq, sf, fmt)
    bad = x.clone()
    bad[M - 1, 77] = float("nan")
    y = fg.gemv_fp4(bad, wq, sf, fmt)
    assert torch.isnan(y[M - 1]).all() and torch.equal(y[: M - 1], clean[: M - 1])
    bad[M - 1, 77] = float("-inf")
    y = fg.gemv_fp4(bad, wq, sf, fmt)
    w = w64[:, 77].to(dev)
    want = torch.where(w > 0, -torch.inf, torch.where(w < 0, torch.inf, torch.nan))     # 0 times infinity
    assert torch.equal(y[: M - 1], clean[: M - 1])
    assert torch.equal(torch.nan_to_num(y[M - 1].float(), nan=3.0), torch.nan_to_num(want.float(), nan=3.0))
    zero = torch.zeros_like(x)
    assert (fg.gemv_fp4(zero, wq, sf, fmt) == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 5, 64), (16, 33, 576)])
def test_outputs_stay_inside_their_buffers(fg, dev, oracle, fmt, M, N, K):
    wq, sf, w64 = _weights(oracle, N, K, fmt, 9, dev)
    x = _x(M, K, torch.float16, 10, dev)
    buf = torch.full((M * N + 4096,), 7.0, dtype=torch.float16, device=dev)
    fg.gemv_fp4(x, wq, sf, fmt, out=buf[: M * N].view(M, N))
    assert (buf[M * N:] == 7.0).all()
    _check(buf[: M * N].view(M, N), x, w64)
    buf.fill_(7.0)
    fg.gated_gemv_fp4(x, wq, sf, wq, sf, fmt, out=buf[: M * N].view(M, N))
    assert (buf[M * N:] == 7.0).all()


def test_no_rows(fg, dev, oracle):
    wq, sf, _ = _weights(oracle, 8, 64, 0, 0, dev)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=dev)
    assert fg.gemv_fp4(x, wq, sf, 0).shape == (0, 8)
    assert fg.gated_gemv_fp4(x, wq, sf, wq, sf, 0).shape == (0, 8)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_weights_from_the_quantizer_other_stream_and_graph(fg, dev, fmt):
    """Weights straight from quantize_fp4; a stream of its own; a captured graph."""
    N, K, M = 136, 512, 3
    w = (torch.randn(N, K, generator=torch.Generator().manual_seed(1)) / 16).to(torch.bfloat16).to(dev)
    wq, sf = fg.quantize_fp4(w, fmt)
    x = _x(M, K, torch.bfloat16, 2, dev)
    y0, h0 = fg.gemv_fp4(x, wq, sf, fmt), fg.gated_gemv_fp4(x, wq, sf, wq, sf, fmt)
    # the 4-bit weights are within half a step of w: 1/4 of the group's largest |w| at most
    assert torch.allclose(y0.double(), x.double() @ w.double().t(), atol=float(x.double().abs().sum(1).max() * w.abs().max() / 4))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y1, h1 = fg.gemv_fp4(x, wq, sf, fmt, stream=side), fg.gated_gemv_fp4(x, wq, sf, wq, sf, fmt, stream=side)
    side.synchronize()
    sx, graph = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, h2 = fg.gemv_fp4(sx, wq, sf, fmt), fg.gated_gemv_fp4(sx, wq, sf, wq, sf, fmt)
    for _ in range(3):
        sx.copy_(x)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(y0, y2) and torch.equal(h0, h1) and torch.equal(h0, h2)
