"""GPU tests of the activations far on the negative side, where the logistic is a subnormal
FP32 number or nearly one: times a large U it is a plain value of H.

Derived bound, relative: sigma(y) = t / (1 + t), t = exp(y).  y is off by a few 2^-24 of itself
(two for the constant and the product, four more for GELU's polynomial), t by 6 |y| 2^-24 and a
few units of its last place, which is 2^-149 where t is subnormal; the slope's sum doubles
that.  One rounding to bf16 follows."""
import math

import pytest
import torch

import gated_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def _gates(act):
    if act == "silu":
        g = [-50.0, -80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -92.0, -94.0, 20.0, 60.0, 88.0, 3.0, -3.0]
    else:
        g = [-5.0, -8.0, -9.5, -9.75, -9.875, -10.0, -10.0625, -10.125, -10.1875, -7.0, -6.0, 9.0, 10.5, 5.0, 3.0, -3.0]
    return torch.tensor(g, dtype=torch.bfloat16)


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_far_negative_gates(fg, dev, M, act):
    K, dtype, size = 8, torch.bfloat16, 2.0 ** 100
    vals = _gates(act).to(dev)
    N = vals.numel()
    x = torch.zeros(M, K, dtype=dtype, device=dev)
    x[:, 0] = 1.0
    wg, wu = torch.zeros(N, K, dtype=dtype, device=dev), torch.zeros(N, K, dtype=dtype, device=dev)
    wg[:, 0], wu[:, 0] = vals, torch.where(vals < 0, size, 1.0).to(dtype)
    h, g, u = fg.gated_f16(x, wg, wu, act, save=True)
    assert torch.equal(g, vals.expand(M, N))
    v = vals.double()
    y = v if act == "silu" else 2.0 * ref.GELU_A * (v + ref.GELU_B * v ** 3)
    t = torch.exp(-y.abs())
    rel = 2.0 * (6.0 * y.abs() + 8.0) * 2.0 ** -24 + 4.0 * 2.0 ** -149 / t
    R, T = ref.unit(dtype)

    def check(got, want, what, more=1.0):
        allowed = want.abs() * (R + 2.0 * rel * more) + T
        off = (got.double() - want).abs() - allowed
        assert (off <= 0).all(), (what, got[0].tolist(), want.tolist())

    check(h, ref.act64(v, act) * wu[:, 0].double(), "h")
    # one token carries the whole gradient, so dWg and dWu are dG and dU themselves
    dh = torch.zeros(M, N, dtype=dtype, device=dev)
    dh[0] = wu[:, 0]
    u1 = torch.ones_like(u)
    _, dwg, dwu = fg.gated_f16_backward(dh, x, wg, wu, g, u1, act)
    d = dh[0].double()
    # a'(g) = s + g s (1 - s) y': the terms' magnitudes over the value say how much cancels
    s = torch.sigmoid(y)
    dy = 1.0 if act == "silu" else 2.0 * ref.GELU_A * (1.0 + 3.0 * ref.GELU_B * v ** 2)
    slope = ref.slope64(v, act)
    cancel = (s + (v * s * (1.0 - s) * dy).abs()) / slope.abs()
    check(dwg[:, 0], d * slope, "dwg", cancel)
    check(dwu[:, 0], d * ref.act64(v, act), "dwu")
    assert math.isfinite(float(h.float().abs().max()))
