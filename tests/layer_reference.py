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


# ------------------------------------------------------------------ MoE layer for a few tokens
def dequant(codes, sf):
    """float64 weights of E4M3 codes [N][K] and block scales [N/128][K/128]."""
    w = codes.view(torch.float8_e4m3fn).double()
    return w * sf.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


# A 128-wide chunk on the tensor cores: eight instructions of sixteen products,
# exact ones; each addend is aligned to the step's largest and keeps at least 24
# bits, so it loses less than 2^-24 of the chunk's sum of magnitudes: 128 2^-24.
# The scales' two products, the chunks' and the warps' sums: at most 32 FP32
# roundings of the same magnitudes.
E_DOT = 2.0 ** -17 + 32 * U


def tiny(w):
    """Where numbers run out of exponents: an FP16 chunk's power of two is at most 2^84, so a value of it is off by up
    to half of FP16's last step, 2^-25 2^-84 = 2^-109, times its weight; and an FP32 rounding near zero is off by
    2^-150 where u times the value is less, which the operations of a product and its sums do 2 K + 64 times at most."""
    return 2.0 ** -109 * w.abs().sum(1) + (2 * w.shape[1] + 64) * 2.0 ** -150


def moe_few_tokens(x, ids, share, wg, sg, wu, su, wd, sd):
    """(y, bound of its error before the last rounding) in float64."""
    x = x.double()
    T, H = x.shape
    y = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    e_y = torch.zeros_like(y)
    E = wu.shape[0]
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e < 0 or e >= E:
                continue
            up = dequant(wu[e], su[e])
            u = up @ x[t]
            e_u = E_DOT * (up.abs() @ x[t].abs()) + tiny(up)
            if wg is None:
                h, e_h = u, e_u
            else:
                gate = dequant(wg[e], sg[e])
                gt = gate @ x[t]
                e_g = E_DOT * (gate.abs() @ x[t].abs()) + tiny(gate)
                silu = gt / (1 + torch.exp(-gt))
                # |silu'| <= 1.1; expf, the sum, the quotient and the product: at most 16 u of h
                h, e_h = silu * u, 1.1 * e_g * (u.abs() + e_u) + silu.abs() * e_u + 16 * U * (silu * u).abs()
            # FP16 with a power-of-two scale for 128 values: half a step, or 2^-40 of the chunk's maximum
            e_h = e_h + 2.0 ** -11 * (h.abs() + e_h)
            e_h = e_h + 2.0 ** -40 * h.abs().view(-1, 128).amax(1).repeat_interleave(128) + 16 * 2.0 ** -150
            down = dequant(wd[e], sd[e])
            w = share[t, j].double()
            y[t] += w * (down @ h)
            e_y[t] += w.abs() * (down.abs() @ e_h + (E_DOT + 8 * U * ids.shape[1]) * (down.abs() @ h.abs()) + tiny(down))
            e_y[t] += 2.0 ** -149
    return y, e_y


# ------------------------------------------------------------------ low-rank adapters
def lora(x, ids, a, b, scaling, base):
    """(out, bound of its error before the last rounding) in float64; ids outside [0, adapters): none."""
    out, e = base.double(), torch.zeros(base.shape, dtype=torch.float64, device=base.device)
    parts = 3 if base.dtype == torch.float32 else 2
    for i in range(a.shape[0]):
        t = torch.nonzero(ids == i)[:, 0]
        if not len(t):
            continue
        s = 1.0 if scaling is None else scaling[i].double()
        A, B, xt = a[i].double(), b[i].double(), x[t].double()
        v = s * (xt @ A.t())
        mag = abs(s) * (xt.abs() @ A.abs().t())
        # a chunk of 64 elements on the tensor cores (64 addends, each losing under 2^-24 of their sum), then at most
        # 64 FP32 additions; the product with s; the BF16 parts
        e_v = (64 + 64 + 1) * U * mag + 2.0 ** (-8 * parts) * v.abs()
        out[t] += v @ B.t()
        vb = v.abs() @ B.abs().t()
        # parts * r addends on the tensor cores (the parts' magnitudes together at most 1 + 2^-7 of v's)
        e[t] += e_v @ B.abs().t() * (1 + 2.0 ** -7) + parts * B.shape[1] * U * (1 + 2.0 ** -6) * vb
    return out, e + U * out.abs()
