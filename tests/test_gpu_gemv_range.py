"""GPU tests of the matrix-vector operators on values far apart: small x beside large x that
meet zero weights, and MXFP4 scales over their whole range.

What is allowed.  Products are exact; sums are FP32, in steps of 16 terms that each may drop
2^-23 of the magnitudes added so far, and a few joins: gamma(K) sum |x w|.  Nothing else: an x
whose weights are zero leaves no trace.  Steps among FP32 subnormals drop at most 2^-149 each.
The output is rounded once."""
import pytest
import torch

import fp4_weights as fp4
import gated_reference as ref

pytestmark = pytest.mark.gpu
FMTS = [0, 1]          # MXFP4, NVFP4


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def _sums(x, w):
    """X W^T in 64 bits, the bound on FP32 sums, sum |x w|."""
    x = x.double()
    mags = x.abs() @ w.abs().t()
    return x @ w.t(), ref.gamma(x.shape[1]) * mags + x.shape[1] * 2.0 ** -149, mags


def _check(got, x, w, what=""):
    R, T = ref.unit(x.dtype)
    y, err, mags = _sums(x, w)
    inside = mags < 2.0 ** 126                 # sums that FP32 holds, whatever their order
    assert inside.any()
    b = err + R * (y.abs() + err) + T
    ref.close(got[inside], y[inside], b[inside], what)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [1, 3, 8, 9, 16])
def test_large_x_on_zero_weights(fg, dev, M, dtype, fmt, gated):
    """One channel of some rows of X is far above the rest, and three weight rows of four are
    zero there: their outputs are those of the other channels."""
    N, K, channel = 52, 832, 300
    gen = torch.Generator(device=dev).manual_seed(M + fmt)
    codes = torch.randint(0, 16, (N, K), generator=gen, device=dev, dtype=torch.uint8)
    zero = torch.arange(N, device=dev) % 4 != 0
    codes[zero, channel] = 8 * (torch.arange(N, device=dev) % 2).to(torch.uint8)[zero]     # plus and minus zero
    lo, hi = (122, 127) if fmt == 0 else (0x14, 0x24)
    scales = torch.randint(lo, hi, (N, K // fp4.GROUP[fmt]), generator=gen, device=dev, dtype=torch.uint8)
    wq, sf = fp4.pack(codes, scales)
    w = fp4.values(codes, scales, fmt)
    base = torch.randn(M, K, generator=gen, device=dev)
    powers = [20, 30, 31, 32, 36, 40, 60, 110] if dtype == torch.bfloat16 else [10, 14]
    for p in powers:
        x = base.clone()
        x[M // 2:, channel] = 2.0 ** p
        x = x.to(dtype)
        if not gated:
            _check(fg.gemv_fp4(x, wq, sf, fmt), x, w, f"2^{p}")
            continue
        h = fg.gated_gemv_fp4(x, wq, sf, wq, sf, fmt)
        g, dg, _ = _sums(x, w)
        want, bound = ref.gate64(g, dg, g, dg, "silu", dtype)
        inside = want.abs() < 2.0 ** 126
        ref.close(h[inside], want[inside], bound[inside], f"2^{p}")


def test_one_beside_a_zero_weight(fg, dev):
    """x = (2^40, 1, 0, ...) against codes (0, 1.0, ...) is 1."""
    codes = torch.zeros((16, 64), dtype=torch.uint8, device=dev)
    codes[:, 1] = 2
    for fmt, one in ((0, 127), (1, 0x38)):
        scales = torch.full((16, 64 // fp4.GROUP[fmt]), one, dtype=torch.uint8, device=dev)
        wq, sf = fp4.pack(codes, scales)
        for p in (0, 20, 31, 32, 40, 100, 127):
            x = torch.zeros((2, 64), dtype=torch.bfloat16, device=dev)
            x[:, 0], x[:, 1] = 2.0 ** p, 1.0
            assert (fg.gemv_fp4(x, wq, sf, fmt) == 1.0).all(), (fmt, p)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 8, 16])
def test_x_over_the_whole_range_of_bf16(fg, dev, M, fmt):
    """Every x of a size of its own, subnormals among them; in each weight row only the x
    below a size of its own meet weights that are not zero."""
    N, K = 64, 768
    gen = torch.Generator(device=dev).manual_seed(M)
    e = torch.randint(-130, 100, (K,), generator=gen, device=dev)
    x = (torch.ldexp(1.0 + torch.rand(M, K, generator=gen, device=dev, dtype=torch.float64), e) *
         torch.where(torch.rand(M, K, generator=gen, device=dev) < 0.5, -1.0, 1.0)).to(torch.bfloat16)
    codes = torch.randint(0, 16, (N, K), generator=gen, device=dev, dtype=torch.uint8)
    limit = torch.linspace(-110, 100, N, device=dev)
    codes[e[None, :] > limit[:, None]] = 0
    scales = torch.full((N, K // fp4.GROUP[fmt]), 127 if fmt == 0 else 0x38, dtype=torch.uint8, device=dev)
    wq, sf = fp4.pack(codes, scales)
    _check(fg.gemv_fp4(x, wq, sf, fmt), x, fp4.values(codes, scales, fmt))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [1, 5, 8, 16])
@pytest.mark.parametrize("K", [256, 320, 1088])
def test_mx_scales_of_any_size_stay_in_their_rows(fg, dev, K, M, dtype):
    """MXFP4 weight rows and groups whose scales lie anywhere in 2^-127 .. 2^127, side by side,
    on rows of X of very different sizes."""
    N = 75
    gen = torch.Generator(device=dev).manual_seed(K + M)
    bytes_ = torch.tensor([0, 1, 3, 20, 40, 62, 63, 64, 65, 100, 127, 150, 190, 191, 192, 193, 220, 245, 252, 254], device=dev)
    own = bytes_[torch.randint(0, len(bytes_), (N, 1), generator=gen, device=dev)]
    near = (own + torch.randint(-3, 4, (N, K // 32), generator=gen, device=dev)).clamp(0, 254)
    any_ = bytes_[torch.randint(0, len(bytes_), (N, K // 32), generator=gen, device=dev)]
    mixed = torch.arange(N, device=dev)[:, None] % 3 == 0          # rows whose groups differ too
    scales = torch.where(mixed, any_, near).to(torch.uint8)
    codes = torch.randint(0, 16, (N, K), generator=gen, device=dev, dtype=torch.uint8)
    wq, sf = fp4.pack(codes, scales)
    w = fp4.values(codes, scales, 0)
    sizes = [0, 125, -120, 60, -60, 100, -100, 30] if dtype == torch.bfloat16 else [0, 10, -10, 5]
    x = torch.randn(M, K, generator=gen, device=dev, dtype=torch.float64)
    for shift in range(len(sizes)):
        e = torch.tensor([sizes[(m + shift) % len(sizes)] for m in range(M)], device=dev)
        xs = torch.ldexp(x, e[:, None]).to(dtype)
        R, T = ref.unit(dtype)
        y, err, mags = _sums(xs, w)
        top = 2.0 ** 126 if dtype == torch.bfloat16 else 2.0 ** 14
        inside = mags < top
        if not inside.any():
            continue
        b = err + R * (y.abs() + err) + T
        ref.close(fg.gemv_fp4(xs, wq, sf, 0)[inside], y[inside], b[inside], f"shift {shift}")


def test_a_neighbours_large_scale(fg, dev):
    """Two weight rows of one tile: scale 2^-100 on x of 2^126 gives what it gives whatever the
    other row's scale; scale 2^-127 on x of about 2^98, beside an x of 2^127 with weight
    zero, keeps the digits of x."""
    codes = torch.zeros((16, 256), dtype=torch.uint8, device=dev)
    scales = torch.full((16, 8), 127, dtype=torch.uint8, device=dev)
    codes[0, :32] = 7                                  # 6.0
    scales[0] = 27
    scales[1] = 200
    wq, sf = fp4.pack(codes, scales)
    x = torch.zeros((1, 256), dtype=torch.bfloat16, device=dev)
    x[0, :32] = 2.0 ** 126
    assert float(fg.gemv_fp4(x, wq, sf, 0)[0, 0]) == 192 * 2.0 ** 26
    codes.zero_()
    codes[2, 1] = 1
    scales[:] = 127
    scales[2] = 0
    wq, sf = fp4.pack(codes, scales)
    x.zero_()
    x[0, 0], x[0, 1] = 2.0 ** 127, 255.0 * 2.0 ** 90
    assert float(fg.gemv_fp4(x, wq, sf, 0)[0, 2]) == 255.0 * 2.0 ** -38


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 7, 16])
def test_zeros_in_x(fg, dev, M, fmt):
    """Rows of X that are mostly zero, of either sign, beside large and small ones: zeros say
    nothing about how far the rest lies apart."""
    N, K = 50, 1088
    gen = torch.Generator(device=dev).manual_seed(M + 20)
    wq, sf, w = fp4.random_matrix(N, K, fmt, 8, dev)
    x = torch.randn(M, K, generator=gen, device=dev)
    x = torch.where(torch.rand(M, K, generator=gen, device=dev) < 0.6, torch.copysign(torch.zeros_like(x), x), x)
    _check(fg.gemv_fp4(x.to(torch.bfloat16), wq, sf, fmt), x.to(torch.bfloat16), w, "zeros")
    small = x * 2.0 ** -40
    small[:, 5] = 1.5
    small[0, 300:] = 0.0
    codes = wq.clone()
    codes[:, 2] &= 0x0F                                  # no weight on column 5
    w[:, 5] = 0.0
    x = small.to(torch.bfloat16)
    _check(fg.gemv_fp4(x, codes, sf, fmt), x, w, "small ones")
    zero = torch.zeros_like(x)
    zero[:, ::3] = -0.0
    assert (fg.gemv_fp4(zero, wq, sf, fmt) == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [2, 16])
def test_non_finite_x_beside_small_x(fg, dev, M, fmt):
    """Infinities and NaN in chunks that also hold x far apart give what the definition gives,
    in their own rows only."""
    N, K = 40, 512
    wq, sf, w = fp4.random_matrix(N, K, fmt, 5, dev)
    x = torch.randn(M, K, generator=torch.Generator(device=dev).manual_seed(1), device=dev).to(torch.bfloat16)
    x[:, 7] = 2.0 ** 50
    clean = fg.gemv_fp4(x, wq, sf, fmt)
    _check(clean, x, w)
    bad = x.clone()
    bad[M - 1, 40] = float("inf")
    y = fg.gemv_fp4(bad, wq, sf, fmt)
    want = torch.where(w[:, 40] > 0, torch.inf, torch.where(w[:, 40] < 0, -torch.inf, torch.nan)).float()
    assert torch.equal(y[: M - 1], clean[: M - 1])
    assert torch.equal(torch.nan_to_num(y[M - 1].float(), nan=3.0), torch.nan_to_num(want, nan=3.0))
    bad[M - 1, 40] = float("nan")
    y = fg.gemv_fp4(bad, wq, sf, fmt)
    assert torch.isnan(y[M - 1]).all() and torch.equal(y[: M - 1], clean[: M - 1])
