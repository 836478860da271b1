"""Plain 64-bit forms of the operators around an FP8 projection, and the error
bounds that the tests compare with.

u = 2^-24 is half a step of FP32 (an operation's relative rounding).  A sum of
n terms in any order is off by at most (n - 1) u times the sum of the terms'
magnitudes; the kernels add along trees, so a bound with the depth of theirs
(at most kDepth additions follow one another on a way through a row's sum)
holds as well and is used where n is large.
"""
from __future__ import annotations

import torch

U = 2.0 ** -24
# additions on the longest way through a row's sum: 16 in a thread, 5 across the
# warp, 7 across the warps and a final product, doubled for the deviations'
# second pass and rounded up
kDepth = 64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ layer norm
def layer_norm(x, gamma, beta, eps):
    """(y, mean, rstd, xh) in float64; gamma/beta may be None."""
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    y = xh if gamma is None else xh * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return y, mean[:, 0], rstd[:, 0], xh


def layer_norm_bound(x, gamma, beta, rstd, xh):
    """Bound of the FP32 y's error.  The mean is off by at most kDepth u mean|x|; xh takes that error and the
    subtraction's times rstd, and rstd's own relative error, which is the variance's: the deviations' errors over
    sigma (the same terms again) and the sum's depth."""
    x = x.double().abs()
    r = rstd[:, None]
    e = kDepth * U * (1 + xh.abs()) * (1 + r * (x.mean(1, keepdim=True) + x))
    if gamma is not None:
        e = e * gamma.double().abs()
    if beta is not None:
        e = e + 2 * U * beta.double().abs()
    return e


def layer_norm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) in float64 from the given statistics."""
    dy, x = dy.double(), x.double()
    mean, r = mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * r
    g = dy if gamma is None else dy * gamma.double()
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def layer_norm_backward_bounds(dy, x, gamma, mean, rstd):
    """Bounds of dx's (before its rounding), dgamma's and dbeta's errors."""
    dy, x = dy.double(), x.double()
    mean, r = mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * r
    g = (dy if gamma is None else dy * gamma.double()).abs()
    e_xh = 4 * U * (r * (x.abs() + mean.abs()) + xh.abs())
    c2 = (g * xh.abs()).mean(1, keepdim=True)
    e_c1 = kDepth * U * g.mean(1, keepdim=True)
    e_c2 = kDepth * U * c2 + (g * e_xh).mean(1, keepdim=True)
    e_dx = r * (8 * U * (g + g.mean(1, keepdim=True) + xh.abs() * c2) + e_c1 + xh.abs() * e_c2 + e_xh * c2)
    M = x.shape[0]
    e_dgamma = (dy.abs() * e_xh).sum(0) + (M + 2) * U * (dy * xh).abs().sum(0)
    e_dbeta = M * U * dy.abs().sum(0)
    return e_dx, e_dgamma, e_dbeta
