"""Layer norm of rows whose mean is thousands of their standard deviation, and of rows of one value: a warp a row, a block
a row, and the streams (test_layer_mean_host.py shows the bounds fail a one-pass variance)."""
import pytest
import torch

import layer_mean_rows as D
import layer_reference as R
from common import load_fp8q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N", [(8, 256), (8, 512), (8, 2048), (8, 7168), (8, 12032), (2370, 1024), (2370, 2048), (2370, 7168)])
def test_large_means_and_constant_rows(fp8q, M, N, dtype):
    x = D.rows(M, N, dtype, M + N, "cuda")
    assert D.ratio(x) > (2000 if dtype == torch.float32 else 500)
    c = torch.tensor(D.CONSTANT[dtype], dtype=dtype).item()
    constant = torch.zeros(M, dtype=torch.bool, device="cuda")
    constant[[1, M - 1]] = True
    x[constant] = c
    y, mean, rstd = fp8q.layer_norm(x, eps=D.EPS)
    want, wm, wr, xh = R.layer_norm(x, None, None, D.EPS)
    e = R.layer_norm_bound(x, None, None, wr, xh)
    tol = e + R.half_step(dtype) * (want.abs() + e)
    assert ((y.double() - want).abs() <= tol)[~constant].all()
    assert ((mean.double() - wm).abs() <= R.kDepth * R.U * x.double().abs().mean(1))[~constant].all()
    assert ((rstd.double() - wr).abs() <= D.rstd_bound(x) * wr)[~constant].all()
    off, low, high = D.constant_bounds(c)
    assert ((mean[constant].double() - c).abs() <= off).all()
    assert ((rstd[constant].double() >= low) & (rstd[constant].double() <= high)).all()
    assert (y[constant].double().abs() <= off * high * (1 + R.half_step(dtype) + 4 * R.U)).all()
    # the backward pass through these statistics
    dy = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dtype)
    dx, dgamma, dbeta = fp8q.layer_norm_backward(dy, x, None, mean, rstd)
    grads = R.layer_norm_backward(dy, x, None, mean, rstd)
    bounds = R.layer_norm_backward_bounds(dy, x, None, mean, rstd)
    assert ((dx.double() - grads[0]).abs() <= bounds[0] + R.half_step(dtype) * (grads[0].abs() + bounds[0])).all()
    for got, w, b in zip((dgamma, dbeta), grads[1:], bounds[1:]):
        assert ((got.double() - w).abs() <= b + R.U * w.abs()).all()
    assert fp8q.fp8q_device_status() == 0
