"""GPU test of queues of dependent calls: each call reads what the one before wrote, into
buffers used again and again, with and without programmatic launches."""
import pytest
import torch

import fp4_weights as fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fg():
    from fine_grained_fp8_persistent_gb300 import binding
    return binding


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


@pytest.mark.parametrize("M", [1, 4, 16, 40, 300])
def test_queue_of_dependent_calls(fg, dev, M):
    """A block applied to its own output in buffers that stay, its 4-bit weights quantized again
    into the same tables between the passes: the same bits whether kernels start early or not."""
    K, N, steps = 512, 1040, 40
    gen = torch.Generator(device=dev).manual_seed(M)
    dt = torch.bfloat16
    wg, wu = (torch.randn(N, K, generator=gen, device=dev).div_(K ** 0.5).to(dt) for _ in range(2))
    wd = [torch.randn(K, N, generator=gen, device=dev).div_(N ** 0.5 / 4).to(dt) for _ in range(2)]
    nk = N // 64 * 64                                     # columns that the 4-bit products read
    x0 = torch.randn(M, K, generator=gen, device=dev).to(dt)

    def run():
        x, h = x0.clone(), torch.empty(M, N, dtype=dt, device=dev)
        hk, y = torch.empty(M, nk, dtype=dt, device=dev), torch.empty(M, K, dtype=dt, device=dev)
        outs = []
        for i in range(steps):
            fg.gated_f16(x, wg, wu, out=h)
            if M <= 16:
                wq, sf = fg.quantize_fp4(wd[i % 2][:, :nk].contiguous(), "nvfp4")
                hk.copy_(h[:, :nk])
                fg.gemv_fp4(hk, wq, sf, "nvfp4", out=y)
            else:
                fg.gemm_f16(h, wd[i % 2], out=y)
            x.copy_(y / (y.float().abs().amax(1, keepdim=True) + 1e-6).to(dt))
            outs.append(y.clone())
        torch.cuda.synchronize()
        return torch.stack(outs)

    before = fg.set_pdl(0)
    try:
        want = run()
        fg.set_pdl(1)
        for _ in range(4):
            assert torch.equal(run(), want)
    finally:
        fg.set_pdl(before)
    assert torch.isfinite(want.float()).all() and fg.check_status()[0] == 0


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("M", [1, 8, 16])
def test_queue_of_matrix_vector_calls(fg, dev, M, fmt):
    """Nothing but matrix-vector kernels, which let the next one start at once: y of one call
    is x of the next, in two buffers taken in turn, clamped between the rounds."""
    K, steps = 1024, 100
    wq, sf, _ = fp4.random_matrix(K, K, fmt, 7, dev)
    x0 = torch.randn(M, K, generator=torch.Generator(device=dev).manual_seed(1), device=dev).to(torch.bfloat16)

    def run():
        a, b = x0.clone(), torch.empty_like(x0)
        for _ in range(steps):
            fg.gemv_fp4(a, wq, sf, fmt, out=b)
            fg.gated_gemv_fp4(b, wq, sf, wq, sf, fmt, out=a)
            fg.gemv_fp4(a, wq, sf, fmt, out=b)
            a, b = b, a
            a.clamp_(-4.0, 4.0)
        torch.cuda.synchronize()
        return a

    before = fg.set_pdl(0)
    try:
        want = run()
        fg.set_pdl(1)
        for _ in range(4):
            assert torch.equal(run(), want)
    finally:
        fg.set_pdl(before)
    assert torch.isfinite(want.float()).all() and (want != 0).any()
