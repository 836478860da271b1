"""The operators around an FP8 projection where calls go wrong: another stream
than the current one, memory past 2^31 elements, calls side by side, and the
largest sizes they take."""
import pytest
import torch

import layer_reference as R
from common import load_fp8q
from test_gpu_lora import make as lora_inputs
from test_gpu_moe_few import layer as expert_layer, routing, tokens

pytestmark = pytest.mark.gpu
HALF = R.half_step(torch.bfloat16)


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


@pytest.mark.parametrize("as_handle", [False, True])
def test_on_a_given_stream(fp8q, as_handle):
    """Every helper's stream argument: inputs produced on that stream late, memory freed at once taken by others'
    work meanwhile, results as on the current stream."""
    side = torch.cuda.Stream()
    arg = side.cuda_stream if as_handle else side
    x0 = tokens(64, 512)
    gamma = torch.rand(512, device="cuda")
    w = expert_layer(4, 512, 256)
    ids, share = routing(64, 2, 4)
    _, a, b, scaling, base, adapter = lora_inputs(64, 3, 16, 512, 256, "bf16")
    rows, _, offsets = fp8q.moe_dispatch_layout(adapter[:, None].contiguous(), 4)

    def everything(x, stream):
        y, mean, rstd = fp8q.layer_norm(x, gamma, stream=stream)
        q, sf, _, _ = fp8q.layer_norm_quant(x, gamma, stream=stream)
        grads = fp8q.layer_norm_backward(y, x, gamma, mean, rstd, stream=stream)
        z = fp8q.moe_few_tokens(x, ids, share, *w, stream=stream)
        out = fp8q.lora_apply(x, rows, offsets, a, b, scaling, base, stream=stream)
        return [y, mean, rstd, q, *grads, z, out]

    want = everything(x0, None)
    torch.cuda.synchronize()
    x = torch.zeros_like(x0)
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)              # the stream is behind the host by some 10 ms
            x.copy_(x0)
        got = everything(x, arg)
        for n in (1 << 10, 1 << 16, 1 << 20):          # the current stream reuses whatever was given back to it
            torch.full((n,), float("nan"), device="cuda")
        side.synchronize()
        for g, e in zip(got, want):
            assert torch.equal(g, e)
        with torch.cuda.stream(side):
            x.zero_()


def test_norm_past_2_31_elements(fp8q):
    """Rows whose offsets pass 32 bits, in the row kernels (odd width) and in the streams (whole vectors)."""
    for N, ld in ((8201, 8208), (4104, 4104)):
        M = (1 << 31) // ld + 40
        x = torch.zeros((M, ld), dtype=torch.bfloat16, device="cuda")
        some = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
        x[some] = torch.randn((5, ld), generator=torch.Generator(device="cuda").manual_seed(N), device="cuda").bfloat16()
        y = torch.empty_like(x)
        mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        fp8q.fp8q_layer_norm(x[:, :N], None, None, 1e-5, y[:, :N], mean, rstd)
        want, _, wr, xh = R.layer_norm(x[some][:, :N], None, None, 1e-5)
        e = R.layer_norm_bound(x[some][:, :N], None, None, wr, xh)
        assert ((y[some][:, :N].double() - want).abs() <= e + HALF * (want.abs() + e)).all()
        assert torch.count_nonzero(y[M // 2 + 1:M - 2]) == 0
        ws = torch.empty(fp8q.lib().fp8q_layer_norm_backward_workspace(M, N), device="cuda")
        dg = torch.empty(N, device="cuda")
        fp8q.fp8q_layer_norm_backward(x[:, :N], x[:, :N], None, mean, rstd, dx=y[:, :N], dgamma=dg, workspace=ws)
        g = R.layer_norm_backward(x[some][:, :N], x[some][:, :N], None, mean[some], rstd[some])
        b = R.layer_norm_backward_bounds(x[some][:, :N], x[some][:, :N], None, mean[some], rstd[some])
        assert ((y[some][:, :N].double() - g[0]).abs() <= b[0] + HALF * (g[0].abs() + b[0])).all()
        # the other rows are zeros: they add exact zeros to the column sums
        assert ((dg.double() - g[1]).abs() <= b[1] + R.U * g[1].abs()).all()
        del x, y


def test_experts_past_2_31_bytes(fp8q):
    """The last of 310 experts of 7168 x 1024 (2.3 GB a matrix), beside the first."""
    w = expert_layer(310, 7168, 1024, seed=4)
    x = tokens(3, 7168)
    ids = torch.tensor([[309, 0], [308, 309], [0, 1]], dtype=torch.int32, device="cuda")
    share = torch.softmax(torch.randn((3, 2), generator=torch.Generator().manual_seed(1)), 1).cuda()
    want, e = R.moe_few_tokens(x, ids, share, *w)
    y = fp8q.moe_few_tokens(x, ids, share, *w)
    assert ((y.double() - want).abs() <= e + HALF * (want.abs() + e)).all()


@pytest.mark.parametrize("T", [2, 40])
def test_adapters_past_2_31_elements(fp8q, T):
    """1020 adapters of rank 128 beside a 16640-wide projection: 2.2e9 values of B; the last adapters' products."""
    n, r, K, N = 1020, 128, 64, 16640
    b = torch.zeros((n, N, r), dtype=torch.bfloat16, device="cuda")
    _, a1, b1, _, base, _ = lora_inputs(T, 3, r, K, N, "bf16", 7)
    x = tokens(T, K)
    a = torch.zeros((n, r, K), dtype=torch.bfloat16, device="cuda")
    for i, adapter in enumerate((0, 1018, 1019)):
        a[adapter], b[adapter] = a1[i], b1[i]
    ids = torch.tensor([0, 1018, 1019], device="cuda")[torch.arange(T, device="cuda") % 3].int()
    if T == 2:
        ids[:] = 1019
    rows, _, offsets = fp8q.moe_dispatch_layout(ids[:, None].contiguous(), 1021)
    out = fp8q.lora_apply(x, rows, offsets, a, b, None, base)
    small = torch.searchsorted(torch.tensor([0, 1018, 1019], device="cuda"), ids.long())
    want, e = R.lora(x, small, a1, b1, None, base)
    assert ((out.double() - want).abs() <= e + HALF * (want.abs() + e)).all()


def test_largest_layer_sizes(fp8q):
    """128 tokens x 8 slots over 1024 experts, rank 128 with 1024 groups, the widest norm."""
    x = tokens(128, 256)
    ids, share = routing(128, 8, 1024)
    w = expert_layer(1024, 256, 128)
    want, e = R.moe_few_tokens(x, ids, share, *w)
    y = fp8q.moe_few_tokens(x, ids, share, *w)
    assert ((y.double() - want).abs() <= e + HALF * (want.abs() + e)).all()
    _, a, b, scaling, base, _ = lora_inputs(3000, 1024, 128, 128, 256, "bf16")
    xs = tokens(3000, 128)
    adapter = torch.randint(0, 1024, (3000,), generator=torch.Generator().manual_seed(0)).int().cuda()
    rows, _, offsets = fp8q.moe_dispatch_layout(adapter[:, None].contiguous(), 1024)
    out = fp8q.lora_apply(xs, rows, offsets, a, b, scaling, base)
    want, e = R.lora(xs, adapter, a, b, scaling, base)
    assert ((out.double() - want).abs() <= e + HALF * (want.abs() + e)).all()
    assert fp8q.fp8q_device_status() == 0


def test_refused_sizes_leave_everything(fp8q):
    """A call past the limits raises before it launches anything."""
    x = tokens(129, 256)
    ids, share = routing(129, 1, 2)
    with pytest.raises(fp8q.FP8QError) as err:
        fp8q.moe_few_tokens(x, ids, share, *expert_layer(2, 256, 128))
    assert err.value.status == fp8q.FP8Q_ERR_UNSUPPORTED
    with pytest.raises(fp8q.FP8QError) as err:
        fp8q.layer_norm(torch.zeros((2, 16392), device="cuda"))
    assert err.value.status == fp8q.FP8Q_ERR_UNSUPPORTED
    with pytest.raises(fp8q.FP8QError) as err:
        fp8q.layer_norm(torch.zeros((2, 257), device="cuda"))          # rows on no 16-byte boundary
    assert err.value.status == fp8q.FP8Q_ERR_ALIGNMENT
    assert fp8q.fp8q_device_status() == 0


def test_two_norms_at_once(fp8q):
    """Forward and backward streams of two calls side by side on two streams, many times: the single calls' bits."""
    xs = [tokens(2400, 1024, s) for s in (1, 2)]
    gamma = torch.rand(1024, device="cuda")
    want = [(fp8q.layer_norm(x, gamma), fp8q.layer_norm_backward(x, x, gamma, *fp8q.layer_norm(x, gamma)[1:])) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                f = fp8q.layer_norm(xs[i], gamma)
                got[i].append((f, fp8q.layer_norm_backward(xs[i], xs[i], gamma, *f[1:])))
    torch.cuda.synchronize()
    for i in (0, 1):
        for f, b in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(f, want[i][0]))
            assert all(torch.equal(p, q) for p, q in zip(b, want[i][1]))
