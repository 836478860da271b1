"""A request whose values overflowed or are NaN does not reach its neighbours: what the layer operators give the other
rows of a batch is bit for bit what they give them beside finite rows, and the row itself shows it."""
import pytest
import torch

from common import load_fp8q
from test_gpu_lora import make, plan
from test_gpu_moe_few import layer, routing, tokens

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


def spoil(t, rows, column):
    t = t.clone()
    for i, r in enumerate(rows):
        t[r, column] = BAD[i % 3]
    return t


# one warp a row, a block a row, the streams
@pytest.mark.parametrize("M,N", [(13, 256), (13, 1024), (2401, 1024)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer_norm(fp8q, M, N, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x, dy = (torch.randn((M, N), generator=g, device="cuda").to(dtype) for _ in range(2))
    gamma, beta = torch.rand(N, generator=g, device="cuda") + 0.5, torch.randn(N, generator=g, device="cuda")
    rows = [0, 5, M - 1]
    good = torch.ones(M, dtype=torch.bool, device="cuda")
    good[rows] = False
    clean = fp8q.layer_norm_quant(x, gamma, beta, keep_y=True)
    dx0, _, _ = fp8q.layer_norm_backward(dy, x, gamma, clean[2], clean[3])
    xs = spoil(x, rows, N - 3)
    got = fp8q.layer_norm_quant(xs, gamma, beta, keep_y=True)
    for i in (0, 2, 3, 4):
        assert torch.equal(got[i][good], clean[i][good])
    assert torch.equal(got[1][:, :M][:, good], clean[1][:, :M][:, good])
    assert got[4][~good].isnan().any(1).all()
    # a spoiled dy reaches its row of dx and every column it weighs in, no other row
    dys = spoil(dy, rows, 2)
    dx, dgamma, dbeta = fp8q.layer_norm_backward(dys, x, gamma, clean[2], clean[3])
    assert torch.equal(dx[good], dx0[good])
    assert dx[~good].isnan().any(1).all()
    assert dbeta[2].isnan() and dbeta[3:].isfinite().all() and dgamma[3:].isfinite().all()


@pytest.mark.parametrize("T,k,E", [(7, 2, 3), (40, 4, 6), (100, 8, 12)])
@pytest.mark.parametrize("gated", [True, False])
def test_moe(fp8q, T, k, E, gated):
    w = layer(E, 384, 256, gated, seed=T)
    ids, share = routing(T, k, E, T)
    x = tokens(T, 384, T)
    rows = [0, T // 2, T - 1]
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[rows] = False
    clean = fp8q.moe_few_tokens(x, ids, share, *w)
    got = fp8q.moe_few_tokens(spoil(x, rows, 77), ids, share, *w)
    assert torch.equal(got[good], clean[good])
    assert (~got[~good].isfinite()).any(1).all()
    # a slot that is skipped may hold anything as its share
    skip = ids.clone()
    skip[:, 0] = -1
    want = fp8q.moe_few_tokens(x, skip, share, *w)
    bad = share.clone()
    bad[:, 0] = float("nan")
    assert torch.equal(fp8q.moe_few_tokens(x, skip, bad, *w), want)
    assert fp8q.fp8q_device_status() == 0


# a token a group with short rows of B, few tokens a group, and many
@pytest.mark.parametrize("T,n,r", [(7, 7, 16), (6, 4, 16), (30, 4, 24), (300, 4, 8), (300, 3, 40), (300, 2, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lora(fp8q, T, n, r, dtype):
    x, a, b, scaling, base, ids = make(T, n, r, 520, 264, dtype, seed=T + r)
    ids[0], ids[T // 2], ids[T - 1] = 0, 1, 0
    offs = plan(fp8q, ids, n + 1)
    rows = [0, T // 2, T - 1]
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[rows] = False
    clean = fp8q.lora_apply(x, *offs, a, b, scaling, base)
    got = fp8q.lora_apply(spoil(x, rows, 519), *offs, a, b, scaling, base)
    assert torch.equal(got[good], clean[good])
    assert (~got[~good].isfinite()).any(1).all()
    # an adapter gone bad spoils its own tokens only
    sick = a.clone()
    sick[0, r - 1, 3] = float("nan")
    got = fp8q.lora_apply(x, *offs, sick, b, scaling, base)
    assert torch.equal(got[ids != 0], clean[ids != 0])
    assert got[ids == 0].isnan().all()
    sick = b.clone()
    sick[0, 7, r - 1] = float("nan")
    got = fp8q.lora_apply(x, *offs, a, sick, scaling, base)
    keep = torch.ones_like(clean, dtype=torch.bool)
    keep[:, 7] = ids != 0
    assert torch.equal(got[keep], clean[keep])
    assert got[ids == 0, 7].isnan().all()
    assert fp8q.fp8q_device_status() == 0
