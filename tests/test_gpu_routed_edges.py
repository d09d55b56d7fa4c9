"""GPU tests of the routing at the borders of its forms and of 32 bits, and of the bits of
dispatch_fp8 against their definition."""
import numpy as np
import pytest
import torch

import routed_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


# ----------------------------------------------------------------- dispatch_fp8
@pytest.mark.parametrize("T,k,G,K,Mmax", [(64, 8, 32, 7168, 256), (777, 3, 5, 1152, 0), (300, 2, 9, 640, 0)])
def test_fp32_scales_are_the_nearest_and_codes_the_nearest_of_them(fg, dev, T, k, G, K, Mmax):
    """The scale of a group is amax / 448 rounded once, and a code is an E4M3 value nearest to
    x / scale.  In 64 bits: a quotient of an 8-bit significand by 7 * 2^6 is periodic in three
    bits, so no double rounding can move it.  x / scale is rounded to FP32 before it is rounded to
    E4M3, so a code may be off by half a step and 2^-24 of the quotient."""
    ids = ref.random_ids(T, k, G, 5, 0.2)
    gen = torch.Generator().manual_seed(6)
    x = torch.randn(T, K, generator=gen)
    x[:, torch.randint(0, K, (2,), generator=gen)] *= 20.0
    x = x.bfloat16()
    groups = x.double().view(T, K // 128, 128)
    scale = (groups.abs().amax(-1) / 448.0).float()         # both roundings are to nearest
    r = fg.route_masked(ids.to(dev), G, Mmax) if Mmax else fg.route_contiguous(ids.to(dev), G)
    xq, sfa = fg.dispatch_fp8(x.to(dev), r, "f32")
    again = fg.dispatch_fp8(x.to(dev), r, "f32")
    src = r.src.cpu().long()
    own = torch.nonzero(src >= 0).view(-1)
    token = src[own] // k
    codes = xq.view(-1, K).cpu()[own]
    assert torch.equal(codes, again[0].view(-1, K).cpu()[own])
    table = sfa.cpu()
    got = table[own // Mmax, :, own % Mmax] if Mmax else table[:, own].t()
    assert torch.equal(got, scale[token])
    exact = (groups / scale.double().unsqueeze(-1)).view(T, K)[token]
    value = codes.view(torch.float8_e4m3fn).double()
    # the step of E4M3 at a quotient: 2^-3 of its power of two, 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(exact.abs().clamp(min=2.0 ** -6)))) * 2.0 ** -3
    assert ((value - exact).abs() <= step / 2 + 2.0 ** -24 * exact.abs()).all()
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_infinities_and_nans_as_quantize_has_them(fg, dev, fmt):
    """The bits of quantize_1x128 for groups with infinities, NaN and both, and for those beside them."""
    T, k, G, K = 12, 2, 3, 512
    ids = ref.random_ids(T, k, G, 8)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(9))
    x[1, 5], x[2, 130], x[3, 300] = float("inf"), float("-inf"), float("nan")
    x[4, :128] = float("nan")
    x[5, 0], x[5, 1] = float("inf"), float("nan")
    x[6] = float("inf")
    x = x.bfloat16().to(dev)
    codes, table = (t.cpu() for t in fg.quantize_1x128(x, fmt))
    r = fg.route_contiguous(ids.to(dev), G)
    xq, sfa = (t.cpu() for t in fg.dispatch_fp8(x, r, fmt))
    src = r.src.cpu().long()
    own = torch.nonzero(src >= 0).view(-1)
    assert torch.equal(xq[own], codes[src[own] // k])
    assert torch.equal(sfa[:, own].view(torch.int32), table[:, src[own] // k].view(torch.int32))


# ----------------------------------------------------------------- routing
def test_segments_of_two_thousand_million_rows(fg, dev):
    """One group whose entries and segment together pass 2^31: its padded size does not."""
    n, M = 2000, 0x7FFFFFFF - 1023
    ids = torch.zeros(n, dtype=torch.int32, device=dev)
    ids[7] = -1
    r = fg.route_contiguous(ids, 1, align=M)
    assert fg.route_rows(n, 1, 1, M) == M == r.src.shape[0]
    assert r.starts.tolist() == [0, M] and r.counts.tolist() == [n - 1]
    at = torch.nonzero(ids == 0).view(-1).int()
    assert torch.equal(r.rows.view(-1)[at.long()], torch.arange(n - 1, device=dev, dtype=torch.int32)) and int(r.rows[7, 0]) == -1
    assert torch.equal(r.src[: n - 1], at) and not r.m_indices[: n - 1].any()
    for t in (r.src, r.m_indices):
        for piece in t[n - 1:].split(1 << 28):
            assert (piece == -1).all()


# Lists of up to 512 entries take one CTA (sixteen times where entries and rows are more than
# 4096), up to 16384 eight of them in a cluster, longer ones sixteen.
@pytest.mark.parametrize("n", [1, 5, 511, 512, 513, 3000, 16383, 16384, 16385])
@pytest.mark.parametrize("G,align", [(7, 1), (32, 128), (1000, 16)])
def test_lists_at_the_borders_of_the_forms(fg, dev, n, G, align):
    ids = ref.random_ids(n, 1, G, n + G, 0.1, 0.2)
    M = fg.route_rows(n, 1, G, align)
    for rows in (M, M + (4096 + align - 1) // align * align):
        r = fg.route_contiguous(ids.to(dev), G, align, M=rows)
        for got, want, name in zip(r[:5], ref.route(ids.numpy(), G, align, rows), r._fields):
            assert np.array_equal(got.cpu().numpy(), want), (rows, name)
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("T,k,G,Mmax", [(64, 8, 32, 256), (1, 8, 32, 256), (3, 1, 32, 256), (63, 8, 5, 1000), (64, 8, 32, 3)])
def test_few_entries_for_many_slots(fg, dev, T, k, G, Mmax):
    """A decode step: few entries, which sixteen CTAs count and place, some with fewer warps' shares
    than there are CTAs."""
    for absent in (0.0, 0.3, 1.0):
        ids = ref.random_ids(T, k, G, T + k, absent, 0.1)
        for given in (ids, ids.long()):
            r = fg.route_masked(given.to(dev), G, Mmax)
            want = ref.route(ids.numpy(), G, 1, G * Mmax, Mmax)
            for got, w, name in ((r.rows, want[0], "rows"), (r.src, want[1], "src"), (r.counts, want[3], "counts")):
                assert np.array_equal(got.cpu().numpy(), w), name
    assert fg.check_status()[0] == 0
