"""4-bit weight matrices made directly from codes and scale bytes, in the layout that
quantize_fp4 writes, and their values in 64 bits."""
from __future__ import annotations

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
GROUP = {0: 32, 1: 16}     # columns per scale: MXFP4, NVFP4


def pack(codes: torch.Tensor, scales: torch.Tensor):
    """(wq uint8 (N, K/2), sf int32 (words, N padded to 4)) of codes (N, K) and scale bytes
    (N, K / group), both uint8."""
    N, groups = scales.shape
    wq = (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()
    words = (groups + 3) // 4
    per_row = torch.zeros((N, words * 4), dtype=torch.uint8, device=codes.device)
    per_row[:, :groups] = scales
    sf = torch.zeros((words, (N + 3) // 4 * 4, 4), dtype=torch.uint8, device=codes.device)
    sf[:, :N] = per_row.view(N, words, 4).permute(1, 0, 2)
    return wq, sf.view(torch.int32).squeeze(-1)


def values(codes: torch.Tensor, scales: torch.Tensor, fmt: int) -> torch.Tensor:
    """The matrix in 64 bits."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    if fmt == 0:
        s = torch.ldexp(torch.ones((), dtype=torch.float64, device=codes.device), scales.int() - 127)
    else:
        s = scales.view(torch.float8_e4m3fn).double()
    N, K = codes.shape
    return (table[codes.long()].view(N, -1, GROUP[fmt]) * s.unsqueeze(-1)).view(N, K)


def random_matrix(N: int, K: int, fmt: int, seed: int, device):
    """(wq, sf, values) with random codes and scales around 1/8."""
    gen = torch.Generator(device=device).manual_seed(seed)
    codes = torch.randint(0, 16, (N, K), generator=gen, device=device, dtype=torch.uint8)
    lo, hi = (122, 127) if fmt == 0 else (0x14, 0x24)
    scales = torch.randint(lo, hi, (N, K // GROUP[fmt]), generator=gen, device=device, dtype=torch.uint8)
    return *pack(codes, scales), values(codes, scales, fmt)
