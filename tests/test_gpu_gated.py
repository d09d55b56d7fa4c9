"""GPU tests of gated_f16 and gated_f16_backward against their definition in 64 bits."""
import pytest
import torch

import gated_reference as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]
# one token, row counts on both sides of every tile height and of the few-token form;
# inner and hidden sizes down to 8 and past every tile width by 8
SHAPES = [(1, 8, 8), (1, 264, 1032), (2, 40, 7168), (3, 520, 64), (8, 136, 200), (15, 24, 4104), (16, 128, 256), (17, 16, 72),
          (31, 72, 520), (64, 256, 128), (65, 8, 2056), (127, 1000, 64), (128, 264, 8), (129, 136, 136), (255, 24, 1032),
          (256, 512, 256), (257, 264, 264), (513, 1032, 520), (1300, 776, 328)]


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def _inputs(M, N, K, dtype, seed, dev):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=gen)
    x[:, :: max(1, K // 3)] *= 8.0
    wg, wu = (torch.randn(N, K, generator=gen) / K ** 0.5 for _ in range(2))
    return tuple(t.to(dtype).to(dev) for t in (x, wg, wu))


def _grad_inputs(M, N, K, dtype, seed, dev):
    x, wg, wu = _inputs(M, N, K, dtype, seed, dev)
    g, u = (x.double() @ wg.double().t()).to(dtype), (x.double() @ wu.double().t()).to(dtype)
    dh = (torch.randn(M, N, generator=torch.Generator().manual_seed(seed + 1)) * 0.1).to(dtype).to(dev)
    return dh, x, wg, wu, g, u


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(fg, dev, M, N, K, dtype, act):
    x, wg, wu = _inputs(M, N, K, dtype, M + N + K, dev)
    want, bound = ref.forward64(x, wg, wu, act)
    h, g, u = fg.gated_f16(x, wg, wu, act, save=True)
    for got, w, b, what in zip((h, g, u), want, bound, "hgu"):
        ref.close(got, w, b, what)
    only = fg.gated_f16(x, wg, wu, act)
    assert torch.equal(only, h)                       # with and without keeping G, U, and run to run
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_backward(fg, dev, M, N, K, dtype, act):
    dh, x, wg, wu, g, u = _grad_inputs(M, N, K, dtype, M + N + K, dev)
    want, bound = ref.backward64(dh, x, wg, wu, g, u, act)
    got = fg.gated_f16_backward(dh, x, wg, wu, g, u, act)
    for t, w, b, what in zip(got, want, bound, ("dx", "dwg", "dwu")):
        ref.close(t, w, b, what)
    again = fg.gated_f16_backward(dh, x, wg, wu, g, u, act)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tile", ["2x256", "1x128", "1x64"])
@pytest.mark.parametrize("M,N,K", [(20, 40, 72), (300, 520, 200), (640, 1304, 136)])
def test_every_tile(fg, dev, monkeypatch, M, N, K, tile, dtype):
    """Each tile shape, whatever the launcher would choose."""
    dh, x, wg, wu, g, u = _grad_inputs(M, N, K, dtype, 11, dev)
    monkeypatch.setenv("FGF8_FORCE_TILE", tile)
    got = fg.gated_f16(x, wg, wu, "silu", save=True)
    assert fg.last_tile() == f"f16 gated {tile}"
    for t, w, b, what in zip(got, *ref.forward64(x, wg, wu, "silu"), "hgu"):
        ref.close(t, w, b, what)
    got = fg.gated_f16_backward(dh, x, wg, wu, g, u)
    assert fg.last_tile() == f"f16 gated_grad {tile}"
    for t, w, b, what in zip(got, *ref.backward64(dh, x, wg, wu, g, u, "silu"), ("dx", "dwg", "dwu")):
        ref.close(t, w, b, what)
    assert fg.check_status()[0] == 0


@pytest.mark.parametrize("act", ref.ACTS)
def test_backward_against_differences(fg, dev, act):
    """Along random directions, the gradients agree with central differences of the 64-bit
    loss sum(dH * H).  Off by the gradients' own bounds and by the rounding of the kept G
    and U: dG moves by |dH| (|U| 1.2 R |G| + 1.13 R |U|), dU by |dH| 1.13 R |G| (slopes
    are below 1.13, their derivatives below 1.2)."""
    M, N, K, dtype = 6, 24, 32, torch.float16
    x, wg, wu = _inputs(M, N, K, dtype, 5, dev)
    dh = (torch.randn(M, N, generator=torch.Generator().manual_seed(6))).to(dtype).to(dev)
    _, g, u = fg.gated_f16(x, wg, wu, act, save=True)
    got = [t.double() for t in fg.gated_f16_backward(dh, x, wg, wu, g, u, act)]
    R, _ = ref.unit(dtype)
    _, bounds = ref.backward64(dh, x, wg, wu, g, u, act)
    a = dh.double().abs()
    gm, um = g.double().abs(), u.double().abs()
    ddg, ddu = a * (um * 1.2 * R * gm + 1.13 * R * um), a * 1.13 * R * gm
    xd, gd, ud = x.double(), wg.double(), wu.double()
    more = (ddg @ gd.abs() + ddu @ ud.abs(), ddg.t() @ xd.abs(), ddu.t() @ xd.abs())

    def loss(p, q, r):
        return float((dh.double() * ref.act64(p @ q.t(), act) * (p @ r.t())).sum())

    gen = torch.Generator().manual_seed(7)
    for _ in range(8):
        v = [torch.randn(t.shape, generator=gen, dtype=torch.float64).to(dev) for t in got]
        e = 1e-5
        slope = (loss(xd + e * v[0], gd + e * v[1], ud + e * v[2]) - loss(xd - e * v[0], gd - e * v[1], ud - e * v[2])) / (2 * e)
        mine = sum(float((t * d).sum()) for t, d in zip(got, v))
        allowed = sum(float(((b + m) * d.abs()).sum()) for b, m, d in zip(bounds, more, v))
        assert abs(mine - slope) <= allowed + 1e-6 * abs(slope), (mine, slope, allowed)


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (5, 264, 136), (200, 136, 264)])
def test_outputs_stay_inside_their_buffers(fg, dev, M, N, K):
    """Outputs at the front of larger buffers: nothing past their end is written."""
    def room(*shape):
        n = shape[0] * shape[1]
        buf = torch.full((n + 4096,), 7.0, dtype=torch.bfloat16, device=dev)
        return buf, buf[:n].view(shape), n
    dh, x, wg, wu, g, u = _grad_inputs(M, N, K, torch.bfloat16, 1, dev)
    bufs = [room(M, N) for _ in range(3)]
    fg.gated_f16(x, wg, wu, out=bufs[0][1], g=bufs[1][1], u=bufs[2][1])
    grads = [room(M, K), room(N, K), room(N, K)]
    ws = torch.full((fg.gated_backward_ws_bytes(M, N) + 4096,), 9, dtype=torch.uint8, device=dev)
    fg.gated_f16_backward(dh, x, wg, wu, g, u, dx=grads[0][1], dwg=grads[1][1], dwu=grads[2][1], workspace=ws)
    torch.cuda.synchronize()
    for buf, _, n in bufs + grads:
        assert (buf[n:] == 7.0).all()
    assert (ws[fg.gated_backward_ws_bytes(M, N):] == 9).all()
    want, bound = ref.forward64(x, wg, wu, "silu")
    ref.close(bufs[0][1], want[0], bound[0])


@pytest.mark.parametrize("M", [1, 4, 16, 40, 300])
def test_non_finite_rows_stay_to_themselves(fg, dev, M):
    """A token with a NaN gives NaN in its own row of H and dX only; every weight gradient
    then has one, as by the formula.  An infinite token gives what the formula gives."""
    N, K = 72, 136
    x, wg, wu = _inputs(M, N, K, torch.bfloat16, 3, dev)
    clean = fg.gated_f16(x, wg, wu)
    bad = x.clone()
    bad[M - 1, 5] = float("nan")
    h = fg.gated_f16(bad, wg, wu)
    assert torch.isnan(h[M - 1]).all() and torch.equal(h[: M - 1], clean[: M - 1])
    bad[M - 1, 5] = float("inf")
    h, g, u = fg.gated_f16(bad, wg, wu, save=True)
    inf = float("inf")
    assert torch.equal(h[: M - 1], clean[: M - 1])
    assert torch.equal(g[M - 1].float(), torch.where(wg[:, 5] > 0, inf, -inf))
    up = wg[:, 5] > 0                                    # a(inf) = inf, times an infinite U
    assert torch.equal(h[M - 1][up].float(), torch.where(wu[:, 5] > 0, inf, -inf)[up])
    dh, x, wg, wu, g, u = _grad_inputs(M, N, K, torch.bfloat16, 4, dev)
    good = fg.gated_f16_backward(dh, x, wg, wu, g, u)
    dh[M - 1, 9] = float("nan")
    dx, dwg, dwu = fg.gated_f16_backward(dh, x, wg, wu, g, u)
    assert torch.isnan(dx[M - 1]).all() and torch.equal(dx[: M - 1], good[0][: M - 1])
    rows = torch.arange(N, device=dev) != 9
    assert torch.isnan(dwg[9]).all() and torch.equal(dwg[rows], good[1][rows]) and torch.equal(dwu[rows], good[2][rows])


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("M", [1, 130])
def test_far_gates(fg, dev, act, M):
    """Gates far on either side of 0, to the type's largest finite value: a(g) is g or 0,
    the slope 1 or 0, with no NaN from an overflow on the way."""
    dtype, K = torch.bfloat16, 8
    vals = torch.tensor([-3e38, -1e20, -1e4, -120.0, -89.0, -30.0, 0.0, 30.0, 89.0, 120.0, 1e4, 1e20, 3e38, -0.5, 0.5, 2.0], dtype=dtype)
    N = vals.numel()
    x = torch.zeros(M, K, dtype=dtype, device=dev)
    x[:, 0] = 1.0
    wg = torch.zeros(N, K, dtype=dtype, device=dev)
    wg[:, 0] = vals.to(dev)
    wu = torch.zeros_like(wg)
    wu[:, 0] = 0.5
    h, g, u = fg.gated_f16(x, wg, wu, act, save=True)
    want, bound = ref.forward64(x, wg, wu, act)
    ref.close(h, want[0], bound[0])
    assert torch.equal(g, vals.to(dev).expand(M, N))
    dh = torch.full((M, N), 0.25, dtype=dtype, device=dev)
    dh[:, vals.to(dev).float().abs() > 1e30] = 0.0          # keeps the sums finite; 0 times a finite slope is 0
    dx, dwg, dwu = fg.gated_f16_backward(dh, x, wg, wu, g, u, act)
    want, bound = ref.backward64(dh, x, wg, wu, g, u, act)
    ref.close(dwg, want[1], bound[1], "dwg")
    ref.close(dwu, want[2], bound[2], "dwu")


def test_no_tokens(fg, dev):
    x = torch.empty(0, 64, dtype=torch.float16, device=dev)
    w = torch.ones(24, 64, dtype=torch.float16, device=dev)
    h, g, u = fg.gated_f16(x, w, w, save=True)
    assert h.shape == g.shape == u.shape == (0, 24)
    dw = [torch.full((24, 64), 3.0, dtype=torch.float16, device=dev) for _ in range(2)]
    dx, dwg, dwu = fg.gated_f16_backward(h, x, w, w, g, u, dwg=dw[0], dwu=dw[1])
    assert dx.shape == (0, 64) and (dwg == 0).all() and (dwu == 0).all()


@pytest.mark.parametrize("M", [2, 300])
def test_other_stream_and_graph(fg, dev, M):
    """On a stream of its own, and captured into a CUDA graph and replayed on new inputs."""
    N, K = 264, 520
    dh, x, wg, wu, g, u = _grad_inputs(M, N, K, torch.bfloat16, 8, dev)
    h0 = fg.gated_f16(x, wg, wu)
    d0 = fg.gated_f16_backward(dh, x, wg, wu, g, u)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    h1 = fg.gated_f16(x, wg, wu, stream=side)
    d1 = fg.gated_f16_backward(dh, x, wg, wu, g, u, stream=side)
    side.synchronize()
    assert torch.equal(h0, h1) and all(torch.equal(a, b) for a, b in zip(d0, d1))
    sx, graph = torch.zeros_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h2 = fg.gated_f16(sx, wg, wu)
        d2 = fg.gated_f16_backward(dh, sx, wg, wu, g, u)
    for _ in range(3):
        sx.copy_(x)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h0, h2) and all(torch.equal(a, b) for a, b in zip(d0, d2))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_feed_forward_example(fg, dev, fmt):
    """The example trains (its loss falls by half at least) and serves in 4 bits: each of three
    matrices rounds to within a quarter of its groups' steps, about 0.1 of a weight."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, rel = example.main(["--tokens", "256", "--hidden", "512", "--inter", "1024", "--steps", "12", "--fmt", fmt])
    assert losses[-1] < 0.5 * losses[0]
    assert rel < 0.35
