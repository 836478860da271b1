"""The operators around an FP8 projection run together, as a decoding step runs
them, and a training step's norm with its projection and gradients: every stage
against the 64-bit formula of what it was given, and the whole chain captured in
a graph against the direct calls."""
import numpy as np
import pytest
import torch

import layer_reference as R
from common import check_gemm, load_fp8q
from test_gpu_lora import make as lora_inputs
from test_gpu_moe_few import layer as expert_layer, routing

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


def setup(fp8q, T, H=512, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"x": torch.randn((T, H), generator=g, device="cuda").bfloat16()}
    for i in (1, 2):
        s[f"gamma{i}"] = 1 + 0.1 * torch.randn(H, generator=g, device="cuda")
        s[f"beta{i}"] = 0.1 * torch.randn(H, generator=g, device="cuda")
    w = (0.02 * torch.randn((H, H), generator=g, device="cuda")).bfloat16()
    s["wq"], s["ws"] = fp8q.quant_w_128x128(w)
    _, s["a"], s["b"], s["scaling"], _, ids = lora_inputs(T, 3, 16, H, H, "bf16", seed)
    s["adapter"] = ids
    s["rows"], _, s["offsets"] = fp8q.moe_dispatch_layout(ids[:, None].contiguous(), 4)
    s["ids"], s["share"] = routing(T, 2, 5, seed)
    s["experts"] = expert_layer(5, H, 256)
    return s


def step(fp8q, s):
    """norm -> FP8 projection with adapters -> norm -> expert layer."""
    x = s["x"]
    q, sf, mean, rstd, y = fp8q.layer_norm_quant(x, s["gamma1"], s["beta1"], EPS, keep_y=True)
    base = torch.empty_like(x)
    fp8q.fp8q_gemm_blockscaled(q, sf, s["wq"], s["ws"], fp8q.FP8Q_SFB_BLOCK128, base)
    h = fp8q.lora_apply(y, s["rows"], s["offsets"], s["a"], s["b"], s["scaling"], base)
    z, _, _ = fp8q.layer_norm(h, s["gamma2"], s["beta2"], EPS)
    return q, sf, y, base, h, z, fp8q.moe_few_tokens(z, s["ids"], s["share"], *s["experts"])


@pytest.mark.parametrize("T", [1, 7, 100])
def test_decoding_step(fp8q, T):
    s = setup(fp8q, T)
    q, sf, y, base, h, z, out = step(fp8q, s)
    assert fp8q.fp8q_device_status() == 0
    half = R.half_step(torch.bfloat16)
    want, _, wr, xh = R.layer_norm(s["x"], s["gamma1"], s["beta1"], EPS)
    e = R.layer_norm_bound(s["x"], s["gamma1"], s["beta1"], wr, xh)
    assert ((y.double() - want).abs() <= e + half * (want.abs() + e)).all()
    a64 = (q.view(torch.float8_e4m3fn).double().view(T, -1, 128) * sf[:, :T].t().double()[:, :, None]).view(T, -1)
    exact = (a64 @ R.dequant(s["wq"], s["ws"]).t()).cpu().numpy()
    rounded = torch.from_numpy(exact).bfloat16().double().numpy()
    check_gemm(base.double().cpu().numpy(), exact, rounded)
    want, e = R.lora(y, s["adapter"], s["a"], s["b"], s["scaling"], base)
    assert ((h.double() - want).abs() <= e + half * (want.abs() + e)).all()
    want, _, wr, xh = R.layer_norm(h, s["gamma2"], s["beta2"], EPS)
    e = R.layer_norm_bound(h, s["gamma2"], s["beta2"], wr, xh)
    assert ((z.double() - want).abs() <= e + half * (want.abs() + e)).all()
    want, e = R.moe_few_tokens(z, s["ids"], s["share"], *s["experts"])
    assert ((out.double() - want).abs() <= e + half * (want.abs() + e)).all()
    assert np.isfinite(out.float().cpu().numpy()).all()


def test_decoding_step_captured(fp8q):
    """The whole step as one graph, replayed for new tokens, routes and adapters."""
    s = setup(fp8q, 9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(fp8q, s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(fp8q, s)
    for seed in (1, 2, 3):
        new = setup(fp8q, 9, seed=seed)
        for name in ("x", "rows", "offsets", "ids", "share"):
            s[name].copy_(new[name])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step(fp8q, s)):
            # the scales' padding columns are nobody's
            assert torch.equal(a[:, :9] if a.dtype == torch.float32 else a, b[:, :9] if b.dtype == torch.float32 else b)


def test_training_step_of_the_norm(fp8q):
    """Forward: norm into FP8 tiles, projection.  Backward: the projection's input gradient (FP8 Dgrad) through the
    norm; dgamma and dbeta as the formulas of that gradient have them."""
    M, H, N = 256, 512, 256
    s = setup(fp8q, M, H)
    x, gamma = s["x"], s["gamma1"]
    w = (0.02 * torch.randn((N, H), generator=torch.Generator().manual_seed(3))).bfloat16().cuda()
    wq, ws, wqt, wst = fp8q.quant_w_128x128(w, transposed=True)
    q, sf, mean, rstd = fp8q.layer_norm_quant(x, gamma, s["beta1"], EPS)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    fp8q.fp8q_gemm_blockscaled(q, sf, wq, ws, fp8q.FP8Q_SFB_BLOCK128, out)
    dq, dsf = fp8q.quant_act_1x128(out)                                  # loss: half the squared output
    dy = torch.empty((M, H), dtype=torch.bfloat16, device="cuda")
    fp8q.fp8q_gemm_blockscaled(dq, dsf, wqt, wst, fp8q.FP8Q_SFB_BLOCK128, dy)
    dx, dgamma, dbeta = fp8q.layer_norm_backward(dy, x, gamma, mean, rstd)
    want = R.layer_norm_backward(dy, x, gamma, mean, rstd)
    bound = R.layer_norm_backward_bounds(dy, x, gamma, mean, rstd)
    assert ((dx.double() - want[0]).abs() <= bound[0] + R.half_step(x.dtype) * (want[0].abs() + bound[0])).all()
    assert ((dgamma.double() - want[1]).abs() <= bound[1] + R.U * want[1].abs()).all()
    assert ((dbeta.double() - want[2]).abs() <= bound[2] + R.U * want[2].abs()).all()
    # Wgrad's operand of the normalised activation comes from the same tiles (the FP8 activation cache)
    qt = torch.empty((H, M), dtype=torch.uint8, device="cuda")
    sft = torch.empty((M // 128, H), device="cuda")
    fp8q.fp8q_requant_1x128_to_128x1(q, sf, qt, sft)
    assert fp8q.fp8q_device_status() == 0
