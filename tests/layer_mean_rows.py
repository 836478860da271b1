"""Rows whose mean is thousands of their standard deviation, and rows of one value, with bounds that a variance formed as
E[x^2] - mean^2 in FP32 breaks."""
from __future__ import annotations

import torch

import layer_reference as R

EPS = 1e-5
# its square takes 48 bits: an FP32 product of it is rounded
CONSTANT = {torch.float32: 1234.567, torch.bfloat16: 1112.0}


def rows(M, N, dtype, seed, device="cpu"):
    """FP32: 3000 and a deviation of one.  BF16: 1024, and one element in 64 a step (8) higher, a deviation of one too."""
    g = torch.Generator().manual_seed(seed)
    if dtype == torch.float32:
        x = 3000.0 + torch.randn((M, N), generator=g)
    else:
        x = 1024.0 + 8.0 * (torch.rand((M, N), generator=g) < 1 / 64)
        x[:, 0], x[:, 1] = 1024.0, 1032.0                 # no row of one value
    return x.to(dtype).to(device)


def ratio(x):
    x = x.double()
    return (x.mean(1).abs() / x.std(1, correction=0)).min().item()


def rstd_bound(x):
    """Relative bound of rstd's error: the deviations' errors over sigma and the sums' depth (half the variance's)."""
    _, _, r, _ = R.layer_norm(x, None, None, EPS)
    return R.kDepth * R.U * (1 + r * x.double().abs().mean(1))


# A row of one value c, N a multiple of 256 so that every warp's sum of 256 c is exact: the mean takes at most ten
# roundings (the warps' sums joined over at most 4 terms and 5 exchanges, one division), so it is off by 10 u c, every
# deviation as much, rstd between 1 / sqrt(eps + (10 u c)^2) and 1 / sqrt(eps), and y by 10 u c / sqrt(eps).  The
# roundings of these last steps: 4 u.
def constant_bounds(c):
    off = 10 * R.U * c
    least = 1 / (EPS + off ** 2) ** 0.5
    return off, least * (1 - 4 * R.U), EPS ** -0.5 * (1 + 4 * R.U)


def one_pass_rstd(x):
    """What the bounds are there to tell apart: the variance as E[x^2] - mean^2 in FP32."""
    x = x.float()
    mean = x.sum(1) / x.shape[1]
    return ((x * x).sum(1) / x.shape[1] - mean * mean + EPS).rsqrt()
