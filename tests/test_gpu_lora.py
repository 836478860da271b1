"""Low-rank adapters on the GPU against the 64-bit formula, element by element
within the derived bound of layer_reference."""
import pytest
import torch

import layer_reference as R
from common import load_fp8q

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


def make(T, n, r, K, N, dtype, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, (K + 7) // 8 * 8 + pad), generator=g, device="cuda").bfloat16()[:, :K]
    a = (torch.randn((n, r, K), generator=g, device="cuda") / K ** 0.5).bfloat16()
    b = (torch.randn((n, N, r), generator=g, device="cuda") / r ** 0.5).bfloat16()
    scaling = torch.rand(n, generator=g, device="cuda") + 0.5
    base = torch.randn((T, N + pad), generator=g, device="cuda").to(DT[dtype])[:, :N]
    ids = torch.randint(0, n + 1, (T,), generator=g, device="cuda").int()       # n: no adapter
    return x, a, b, scaling, base, ids


def plan(fp8q, ids, groups):
    rows, _, offsets = fp8q.moe_dispatch_layout(ids[:, None].contiguous(), groups)
    return rows, offsets


def check(fp8q, x, ids, a, b, scaling, base, groups=None):
    rows, offsets = plan(fp8q, ids, a.shape[0] + 1 if groups is None else groups)
    want, e = R.lora(x, ids, a, b, scaling, base)
    out = fp8q.lora_apply(x, rows, offsets, a, b, scaling, base)
    tol = e + R.half_step(base.dtype) * (want.abs() + e)
    assert ((out.double() - want).abs() <= tol).all(), ((out.double() - want).abs() / tol).max()
    none = ids >= a.shape[0]
    assert torch.equal(out[none], base[none])
    assert torch.equal(out, fp8q.lora_apply(x, rows, offsets, a, b, scaling, base))
    same = base.clone() if base.is_contiguous() else base
    fp8q.lora_apply(x, rows, offsets, a, b, scaling, same, out=same)            # in place
    assert torch.equal(same, out)
    assert fp8q.fp8q_device_status() == 0
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,n,r,K,N", [(1, 1, 8, 8, 8), (1, 1, 16, 7168, 2048), (3, 2, 16, 72, 40), (5, 5, 24, 200, 264),
                                       (8, 1, 32, 136, 1032), (64, 64, 16, 512, 1024), (33, 4, 40, 1032, 520),
                                       (70, 2, 64, 264, 2056), (200, 3, 8, 1000, 304), (333, 5, 24, 1032, 2056),
                                       (129, 1, 72, 520, 776), (300, 2, 128, 648, 256), (20, 7, 96, 328, 128),
                                       (1, 3, 128, 64, 4096), (600, 1, 48, 128, 512)])
def test_adapters(fp8q, T, n, r, K, N, dtype):
    x, a, b, scaling, base, ids = make(T, n, r, K, N, dtype, T + r)
    if T == n:
        ids = torch.randperm(n).int().cuda()
    check(fp8q, x, ids, a, b, scaling, base)


@pytest.mark.parametrize("T", [3, 90])
def test_shares(fp8q, T):
    """All on one of many, none on any, no scaling, no adapters at all, many empty groups, strided rows."""
    x, a, b, scaling, base, ids = make(T, 6, 16, 256, 512, "bf16", 1, pad=16)
    ids[:] = 4
    check(fp8q, x, ids, a, b, scaling, base.clone())
    check(fp8q, x, ids, a, b, None, base.clone())
    check(fp8q, x, ids, a, b, scaling, base.clone(), groups=1024)
    ids[:] = 6
    assert torch.equal(check(fp8q, x, ids, a, b, scaling, base.clone()), base)
    check(fp8q, x, ids, a[:0], b[:0], scaling[:0], base.clone(), groups=7)
    ids[:] = torch.arange(T, device="cuda") % 7
    check(fp8q, x, ids, a, b, scaling, base)


def test_rows_in_no_group_stay_and_padding_stays(fp8q):
    x, a, b, scaling, base, _ = make(10, 2, 16, 64, 40, "bf16")
    rows = torch.tensor([7, 2, 5, 0, 1, 3, 4, 6, 8, 9], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")         # rows[3:] in no group
    out = torch.full((12, 56), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8q.lora_apply(x, rows, offsets, a, b, scaling, base, out=out[:10, :40])
    ids = torch.full((10,), 2, device="cuda")
    ids[[7, 2]], ids[5] = 0, 1
    want, e = R.lora(x, ids, a, b, scaling, base)
    named = ids < 2
    tol = e + R.half_step(torch.bfloat16) * (want.abs() + e)
    assert ((out[:10, :40].double() - want).abs() <= tol)[named].all()
    assert torch.all(out[:10, :40][~named] == 7.0) and torch.all(out[10:] == 7.0) and torch.all(out[:, 40:] == 7.0)
    assert fp8q.fp8q_device_status() == 0


def test_bad_plans_are_reported(fp8q):
    """Offsets that leave [0, T] are clamped, rows outside [0, T) skipped, both reported; the good rows are right."""
    x, a, b, scaling, base, _ = make(6, 2, 16, 64, 40, "bf16")
    good = torch.arange(6, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    want = fp8q.lora_apply(x, good, offsets, a, b, scaling, base)
    assert fp8q.fp8q_device_status() == 0
    rows = good.clone()
    rows[1], rows[4] = 6, -1
    out = torch.full_like(base, 7.0)
    fp8q.lora_apply(x, rows, offsets, a, b, scaling, base, out=out)
    assert fp8q.fp8q_device_status() & 0xFF == fp8q.FP8Q_ERR_INVALID_ARG
    keep = [0, 2, 3, 5]
    assert torch.equal(out[keep], want[keep]) and torch.all(out[[1, 4]] == 7.0)
    for bad in ([-4, 3, 6], [0, 3, 9], [0, 3, 2]):
        out = fp8q.lora_apply(x, good, torch.tensor(bad, dtype=torch.int32, device="cuda"), a, b, scaling, base)
        assert fp8q.fp8q_device_status() & 0xFF == fp8q.FP8Q_ERR_INVALID_ARG
        assert torch.equal(out[:3], want[:3])
    assert fp8q.fp8q_device_status() == 0


def test_no_tokens(fp8q):
    x, a, b, scaling, base, ids = make(0, 2, 16, 64, 40, "bf16")
    out = fp8q.lora_apply(x, ids, torch.zeros(4, dtype=torch.int32, device="cuda"), a, b, scaling, base)
    assert out.shape == (0, 40)


def test_captured_replayed_and_on_two_streams(fp8q):
    x, a, b, scaling, base, ids = make(40, 5, 16, 512, 1024, "bf16")
    rows, offsets = plan(fp8q, ids, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8q.lora_apply(x, rows, offsets, a, b, scaling, base)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fp8q.lora_apply(x, rows, offsets, a, b, scaling, base)
    x2, _, _, _, base2, ids2 = make(40, 5, 16, 512, 1024, "bf16", 9)
    rows2, offsets2 = plan(fp8q, ids2, 6)
    for dst, src in ((x, x2), (base, base2), (rows, rows2), (offsets, offsets2)):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    want = fp8q.lora_apply(x, rows, offsets, a, b, scaling, base)
    assert torch.equal(out, want)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(fp8q.lora_apply(x, rows, offsets, a, b, scaling, base))
    torch.cuda.synchronize()
    assert all(torch.equal(v, want) for v in got)
