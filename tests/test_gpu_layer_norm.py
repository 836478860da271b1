"""Layer norm on the GPU (forward, 1x128 tiles, backward) against the 64-bit
formulas, element by element within the derived bounds of layer_reference."""
import pytest
import torch

import layer_reference as R
from common import load_fp8q

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


def make(M, N, dtype, seed, offset=0.25, scale=1.5, pad=8):
    g = torch.Generator().manual_seed(seed)
    ld = (N + 7) // 8 * 8 + pad
    x = torch.randn((M, ld), generator=g) * scale + offset
    x[:, ::max(1, N // 3)] *= 20.0
    return x.to(DT[dtype]).cuda()[:, :N]


def params(N, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return ((1 + 0.2 * torch.randn(N, generator=g)).to(DT[dtype]).cuda(),
            (0.3 * torch.randn(N, generator=g)).to(DT[dtype]).cuda())


SHAPES = [(1, 1), (1, 7168), (3, 7), (5, 8), (2, 129), (9, 255), (17, 256), (33, 257), (8, 511), (7, 512), (3, 513),
          (600, 520), (4, 1111), (5, 4096), (3, 4097), (2, 8192), (3, 8193), (1, 16384), (2, 16383), (1200, 1024)]


def check_forward(fp8q, x, gamma, beta, eps=EPS):
    y, mean, rstd = fp8q.layer_norm(x, gamma, beta, eps)
    want, wm, wr, xh = R.layer_norm(x, gamma, beta, eps)
    e = R.layer_norm_bound(x, gamma, beta, wr, xh)
    tol = e + (R.half_step(x.dtype) * (want.abs() + e) if x.dtype == torch.bfloat16 else R.U * want.abs())
    assert ((y.double() - want).abs() <= tol).all()
    assert ((mean.double() - wm).abs() <= R.kDepth * R.U * x.double().abs().mean(1) + 2.0 ** -140).all()
    # rstd's relative error: half the variance's (the deviations' errors over sigma, and the depth)
    rel = R.kDepth * R.U * (1 + wr * x.double().abs().mean(1))
    assert ((rstd.double() - wr).abs() <= rel * wr).all()
    assert fp8q.fp8q_device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_forward(fp8q, M, N, dtype):
    gamma, beta = params(N, "f32", 7 * N + M)
    check_forward(fp8q, make(M, N, dtype, M + N), gamma, beta)


@pytest.mark.parametrize("N", [96, 1000, 9000])
@pytest.mark.parametrize("which", ["none", "gamma", "beta", "bf16"])
def test_forward_parameters(fp8q, N, which):
    gamma, beta = params(N, "bf16" if which == "bf16" else "f32", N)
    if which in ("none", "beta"):
        gamma = None
    if which in ("none", "gamma"):
        beta = None
    check_forward(fp8q, make(5, N, "bf16", N), gamma, beta)
    check_forward(fp8q, make(5, N, "f32", N), gamma, beta)


@pytest.mark.parametrize("N", [200, 2000, 12000])
def test_forward_large_mean_and_constant_rows(fp8q, N):
    """|mean| >> sigma, where E[x^2] - mean^2 would have no digits left; and rows of one value (variance zero)."""
    x = make(6, N, "f32", N, offset=3000.0, scale=0.5)
    x[2] = 7.25
    x[3] = 0.0
    check_forward(fp8q, x, *params(N, "f32", 1))
    y, mean, rstd = fp8q.layer_norm(x, eps=EPS)
    assert torch.equal(mean[2:4].cpu(), torch.tensor([7.25, 0.0]))
    assert torch.equal(y[2:4], torch.zeros_like(y[2:4]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(1, 128), (5, 256), (130, 384), (3, 512), (64, 640), (33, 4096), (7, 7168), (2, 16384)])
def test_tiles(fp8q, M, N, dtype):
    """Scales within y's bound; codes within half an E4M3 step of y / s.  y given too is the same as without tiles."""
    x = make(M, N, dtype, M * N)
    x[M // 2, :128] = 0.5                                       # with gamma = 0 there: an all-zero tile
    gamma, beta = params(N, "f32", N)
    gamma[:128], beta[:128] = 0.0, 0.0
    q, sf, mean, rstd, y = fp8q.layer_norm_quant(x, gamma, beta, EPS, keep_y=True)
    y2, mean2, rstd2 = fp8q.layer_norm(x, gamma, beta, EPS)
    assert torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    want, _, wr, xh = R.layer_norm(x, gamma, beta, EPS)
    e = R.layer_norm_bound(x, gamma, beta, wr, xh)
    amax = want.abs().view(M, N // 128, 128).amax(2)
    e_tile = e.view(M, N // 128, 128).amax(2)
    s = sf[:, :M].t().double()
    s_want = (amax / 448).clamp_min(1e-12)
    assert ((s - s_want).abs() <= e_tile / 448 + 2 * R.U * s_want).all()
    assert torch.all(sf[0, :M] == torch.tensor(1e-12)) and torch.all((q[:, :128] & 127) == 0)
    dec = q.view(torch.float8_e4m3fn).double().view(M, N // 128, 128) * s[:, :, None]
    y64 = want.view(M, N // 128, 128)
    # half a step of a normal code is 2^-4 of the value at most; below 2^-6 the codes lie 2^-9 apart
    step = torch.maximum(y64.abs() * 2.0 ** -4, s[:, :, None] * 2.0 ** -10)
    assert ((dec - y64).abs() <= step * (1 + 2.0 ** -10) + 2 * e.view(M, N // 128, 128)).all()


def test_tiles_feed_the_projection(fp8q):
    """The tiles go into fp8q_gemm_blockscaled as they are, and equal fp8q_quant_act_1x128 of y where y is exact in
    BF16 (gamma = 0: y = beta)."""
    x = make(40, 256, "bf16", 3)
    beta = torch.randn(256, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q, sf, _, _ = fp8q.layer_norm_quant(x, torch.zeros_like(beta), beta, EPS)
    q2, sf2 = fp8q.quant_act_1x128(beta.expand(40, 256).contiguous())
    assert torch.equal(q, q2) and torch.equal(sf[:, :40], sf2[:, :40])


def test_writes_only_the_rows(fp8q):
    """What lies behind a row, and behind the last row, stays."""
    for N in (100, 700, 9001):
        ld = (N + 7) // 8 * 8 + 16
        x = make(3, N, "bf16", 5, pad=16)
        y = torch.full((5, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        fp8q.fp8q_layer_norm(x, None, None, EPS, y[:3, :N])
        assert torch.all(y[:, N:] == 7.0) and torch.all(y[3:] == 7.0) and not torch.any(y[:3, :N] == 7.0)
        dx = torch.full((5, ld), 7.0, dtype=torch.bfloat16, device="cuda")
        _, mean, rstd = fp8q.layer_norm(x)
        fp8q.fp8q_layer_norm_backward(x, x, None, mean, rstd, dx[:3, :N])
        assert torch.all(dx[:, N:] == 7.0) and torch.all(dx[3:] == 7.0)


def check_backward(fp8q, M, N, dtype, gamma, seed=0):
    x = make(M, N, dtype, seed + M + N)
    dy = make(M, N, dtype, seed + 5, offset=0.0, scale=1e-2)
    _, mean, rstd = fp8q.layer_norm(x, gamma, None, EPS)
    dx, dgamma, dbeta = fp8q.layer_norm_backward(dy, x, gamma, mean, rstd)
    want = R.layer_norm_backward(dy, x, gamma, mean, rstd)
    bound = R.layer_norm_backward_bounds(dy, x, gamma, mean, rstd)
    tol = bound[0] + R.half_step(x.dtype) * (want[0].abs() + bound[0]) + 2.0 ** -133
    assert ((dx.double() - want[0]).abs() <= tol).all()
    for got, w, b in zip((dgamma, dbeta), want[1:], bound[1:]):
        assert ((got.double() - w).abs() <= b + R.U * w.abs()).all()
    again = fp8q.layer_norm_backward(dy, x, gamma, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip((dx, dgamma, dbeta), again))
    return dy, x, mean, rstd, dx, dgamma, dbeta


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", SHAPES + [(2000, 100), (700, 7168)])
def test_backward(fp8q, M, N, dtype):
    check_backward(fp8q, M, N, dtype, params(N, "f32", N)[0])


@pytest.mark.parametrize("N", [100, 1000, 9000])
def test_backward_parameters_and_single_outputs(fp8q, N):
    check_backward(fp8q, 9, N, "bf16", None)
    gamma = params(N, "bf16", N)[0]
    dy, x, mean, rstd, dx, dgamma, dbeta = check_backward(fp8q, 9, N, "bf16", gamma)
    only = torch.empty_strided(dx.shape, dx.stride(), dtype=dx.dtype, device="cuda")     # rows 16 bytes apart too
    fp8q.fp8q_layer_norm_backward(dy, x, gamma, mean, rstd, dx=only)
    assert torch.equal(only, dx)
    ws = torch.full((fp8q.lib().fp8q_layer_norm_backward_workspace(9, N),), float("nan"), device="cuda")
    for name, want in (("dgamma", dgamma), ("dbeta", dbeta)):
        out = torch.empty_like(want)
        fp8q.fp8q_layer_norm_backward(dy, x, gamma, mean, rstd, workspace=ws, **{name: out})
        assert torch.equal(out, want)


def test_empty_batch(fp8q):
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = fp8q.layer_norm(x)
    assert y.shape == (0, 256)
    dx, dgamma, dbeta = fp8q.layer_norm_backward(x, x, None, mean, rstd)
    assert torch.all(dgamma == 0) and torch.all(dbeta == 0)


def test_captured_and_replayed(fp8q):
    """Forward and backward in a captured graph, replayed on new inputs, equal the direct calls."""
    x, dy = make(300, 1000, "bf16", 1), make(300, 1000, "bf16", 2, offset=0.0)
    gamma, beta = params(1000, "f32", 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, mean, rstd = fp8q.layer_norm(x, gamma, beta)
        fp8q.layer_norm_backward(dy, x, gamma, mean, rstd)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, mean, rstd = fp8q.layer_norm(x, gamma, beta)
        out = fp8q.layer_norm_backward(dy, x, gamma, mean, rstd)
    x.copy_(make(300, 1000, "bf16", 11))
    g.replay()
    torch.cuda.synchronize()
    y2, mean2, rstd2 = fp8q.layer_norm(x, gamma, beta)
    assert torch.equal(y, y2) and torch.equal(rstd, rstd2)
    assert all(torch.equal(a, b) for a, b in zip(out, fp8q.layer_norm_backward(dy, x, gamma, mean, rstd)))


# many rows: the kernels that stream rows through shared memory, at widths of one and of many blocks an SM, whole and
# odd row counts, and just outside their range
STREAMS = [(2368, 7168), (2371, 520), (4801, 1024), (2400, 4096), (2369, 4104), (2500, 7176), (2367, 1280), (2401, 1027)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", STREAMS)
def test_many_rows(fp8q, M, N, dtype):
    gamma, beta = params(N, "f32", 7 * N + M)
    check_forward(fp8q, make(M, N, dtype, M + N), gamma, beta)
    check_backward(fp8q, M, N, dtype, gamma)


@pytest.mark.parametrize("which", ["none", "bf16"])
def test_many_rows_parameters(fp8q, which):
    gamma, beta = (None, None) if which == "none" else params(2048, "bf16", 1)
    check_forward(fp8q, make(2400, 2048, "bf16", 1), gamma, beta)
    check_forward(fp8q, make(2400, 2048, "f32", 1, offset=2000.0, scale=0.5), gamma, beta)
    check_backward(fp8q, 2400, 2048, "bf16", gamma)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(2370, 7168), (2369, 640), (2368, 1152)])
def test_many_rows_tiles(fp8q, M, N, dtype):
    """The stream's tiles equal those of the same rows in short calls, code for code and scale for scale, up to
    quotients and scales that their statistics' roundings (another order of the same sums) put on the other side of a
    border: within the bounds of y."""
    x = make(M, N, dtype, N)
    gamma, beta = params(N, "f32", N)
    q, sf, mean, rstd, y = fp8q.layer_norm_quant(x, gamma, beta, EPS, keep_y=True)
    want, _, wr, xh = R.layer_norm(x, gamma, beta, EPS)
    e = R.layer_norm_bound(x, gamma, beta, wr, xh)
    tol = e + R.half_step(x.dtype) * (want.abs() + e)
    assert ((y.double() - want).abs() <= tol).all()
    s = sf[:, :M].t().double()
    s_want = (want.abs().view(M, -1, 128).amax(2) / 448).clamp_min(1e-12)
    assert ((s - s_want).abs() <= e.view(M, -1, 128).amax(2) / 448 + 2 * R.U * s_want).all()
    dec = q.view(torch.float8_e4m3fn).double().view(M, -1, 128) * s[:, :, None]
    y64 = want.view(M, -1, 128)
    step = torch.maximum(y64.abs() * 2.0 ** -4, s[:, :, None] * 2.0 ** -10)
    assert ((dec - y64).abs() <= step * (1 + 2.0 ** -10) + 2 * e.view(M, -1, 128)).all()
    only = fp8q.layer_norm_quant(x, gamma, beta, EPS)
    assert torch.equal(only[0], q) and torch.equal(only[1][:, :M], sf[:, :M]) and torch.equal(only[3], rstd)


def test_many_rows_write_only_the_rows(fp8q):
    N, M, ld = 1000, 2400, 1024
    x = make(M, N, "bf16", 5, pad=16)
    y = torch.full((M + 2, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8q.fp8q_layer_norm(x, None, None, EPS, y[:M, :N])
    assert torch.all(y[:, N:] == 7.0) and torch.all(y[M:] == 7.0) and torch.equal(y[:M, :N], fp8q.layer_norm(x)[0])
    dx = torch.full((M + 2, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    _, mean, rstd = fp8q.layer_norm(x)
    fp8q.fp8q_layer_norm_backward(x, x, None, mean, rstd, dx[:M, :N])
    assert torch.all(dx[:, N:] == 7.0) and torch.all(dx[M:] == 7.0)
