"""GPU tests of examples/experts.py: that it runs, and its gradients against 64-bit autograd."""
import os
import sys

import pytest
import torch

import gated_reference

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_runs(capsys):
    import experts
    experts.main(["--tokens", "70", "--experts", "5", "--choices", "3", "--hidden", "256", "--inter", "128", "--steps", "2"])
    assert "projected with adapters: (70, 256)" in capsys.readouterr().out


def test_gradients():
    """Of the five 16-bit roundings on the way (H, G and U, dYs, dG and dU, dXs) each is at most R of
    its value; 8 R of a gradient's largest value holds what they add up to, their signs being as
    mixed as the sums' terms."""
    import experts
    T, E, k, H, N = 90, 4, 2, 64, 48
    dev = torch.device("cuda:0")
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(T, H, generator=gen).half().to(dev)
    wg, wu = ((torch.randn(E, N, H, generator=gen) / H ** 0.5).half().to(dev) for _ in range(2))
    dy = torch.randn(T, N, generator=gen).half().to(dev)
    ids, w = experts.choose(torch.randn(T, E, generator=gen).to(dev), k)
    y, saved = experts.forward(x, ids, w, wg, wu)
    got = (y, *experts.backward(dy, w, wg, wu, saved))
    leaves = [t.double().requires_grad_() for t in (x, w, wg, wu)]
    g = torch.einsum("th,tknh->tkn", leaves[0], leaves[2][ids])
    u = torch.einsum("th,tknh->tkn", leaves[0], leaves[3][ids])
    want = (leaves[1].unsqueeze(-1) * g * torch.sigmoid(g) * u).sum(1)
    want.backward(dy.double())
    R, _ = gated_reference.unit(torch.float16)
    for mine, exact, what in zip(got, (want.detach(), *(t.grad for t in leaves)), ("y", "dx", "dw", "dwg", "dwu")):
        assert float((mine.double() - exact).abs().max()) <= 8 * R * float(exact.abs().max()), what
