"""The few-token MoE layer on the GPU against the 64-bit formula, element by
element within the derived bound of layer_reference."""
import pytest
import torch

import layer_reference as R
from common import load_fp8q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


def weights(g, E, N, K):
    w = (torch.randn((E, N, K), generator=g, device="cuda") * 112).clamp(-448, 448).to(torch.float8_e4m3fn)
    sf = (torch.rand((E, N // 128, K // 128), generator=g, device="cuda") + 0.5) * (0.02 / 112)
    return w.view(torch.uint8), sf


def layer(E, H, I, gated=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wg, sg = weights(g, E, I, H) if gated else (None, None)
    wu, su = weights(g, E, I, H)
    wd, sd = weights(g, E, H, I)
    return wg, sg, wu, su, wd, sd


def tokens(T, H, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(100 + seed)
    x = torch.randn((T, H + pad), generator=g, device="cuda")
    x[:, ::97] *= 20
    return x.bfloat16()[:, :H]


def routing(T, k, E, seed=0):
    g = torch.Generator(device="cuda").manual_seed(200 + seed)
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].int().contiguous()
    return ids, torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1)


def check(fp8q, x, ids, share, w, dtypes=(torch.bfloat16, torch.float32)):
    want, e = R.moe_few_tokens(x, ids, share, *w)
    for dt in dtypes:
        y = fp8q.moe_few_tokens(x, ids, share, *w, out_dtype=dt)
        assert y.dtype == dt
        tol = e + R.half_step(dt) * (want.abs() + e)
        assert ((y.double() - want).abs() <= tol).all(), ((y.double() - want).abs() / tol).max()
        assert torch.equal(y, fp8q.moe_few_tokens(x, ids, share, *w, out_dtype=dt))
    return y


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 1, 128, 128), (1, 2, 5, 256, 128), (2, 3, 4, 128, 384), (8, 2, 3, 640, 256),
                                       (9, 4, 8, 384, 640), (17, 1, 2, 1152, 128), (33, 5, 16, 256, 1280)])
def test_layer(fp8q, T, k, E, H, I, gated):
    ids, share = routing(T, k, E, T)
    check(fp8q, tokens(T, H, T), ids, share, layer(E, H, I, gated, T))
    assert fp8q.fp8q_device_status() == 0


def test_workload_width(fp8q):
    """7168 -> 2048 -> 7168, one token and a few."""
    w = layer(4, 7168, 2048)
    for T in (1, 3, 12):
        ids, share = routing(T, 2, 4, T)
        check(fp8q, tokens(T, 7168, T), ids, share, w)


@pytest.mark.parametrize("T,k,E", [(128, 8, 1024), (128, 8, 8), (128, 1, 1), (64, 16, 20), (100, 3, 2)])
def test_counts_per_expert(fp8q, T, k, E):
    """From experts with one token to one expert with every entry (k may exceed what differs: ids repeat)."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda").int()
    share = torch.randn((T, k), generator=g, device="cuda")
    check(fp8q, tokens(T, 128, E), ids, share, layer(E, 128, 128, True, E), dtypes=(torch.float32,))


def test_skipped_and_repeated_entries(fp8q):
    """Negative ids, rows without any entry, a token naming one expert twice, all skipped."""
    ids, share = routing(6, 4, 7)
    ids[0, 1] = -1
    ids[2] = -5
    ids[3, 0] = ids[3, 1]
    w = layer(7, 256, 256)
    y = check(fp8q, tokens(6, 256), ids, share, w)
    assert torch.all(y[2] == 0)
    assert fp8q.fp8q_device_status() == 0
    ids[:] = -1
    for T in (6, 1):
        y = fp8q.moe_few_tokens(tokens(T, 256), ids[:T].contiguous(), share[:T].contiguous(), *w)
        assert torch.all(y == 0)
    assert fp8q.fp8q_device_status() == 0


def test_bad_expert_id_is_reported(fp8q):
    ids, share = routing(5, 3, 7)
    ids[1, 2] = 7
    check(fp8q, tokens(5, 256), ids, share, layer(7, 256, 128))
    assert fp8q.fp8q_device_status() & 0xFF == fp8q.FP8Q_ERR_INVALID_ARG
    assert fp8q.fp8q_device_status() == 0


def test_magnitudes(fp8q):
    """Values far outside FP16's range, chunks of zeros, and hidden values of every size: the chunks' scales hold them."""
    ids, share = routing(4, 2, 3)
    w = layer(3, 384, 256)
    w[1].mul_(1e-3)                       # gates near zero
    x = tokens(4, 384)
    x[0] *= 2.0 ** 60
    x[1] *= 2.0 ** -60
    x[2, 128:256] = 0
    x[3] = 0
    w[3].mul_(2.0 ** -20)
    y = check(fp8q, x, ids, share, w)
    assert torch.all(y[3] == 0)


def test_every_code(fp8q):
    """One-hot x reads single weights: every E4M3 code (NaN codes aside) comes through exactly, scaled."""
    E, H, I = 1, 256, 256
    codes = torch.arange(256, device="cuda", dtype=torch.int32)
    codes[127], codes[255] = 0, 0
    wu = codes[None, :].expand(I, H).to(torch.uint8).contiguous()[None]         # wu[i][k] = code k
    eye = torch.zeros((1, H, I), device="cuda")
    eye[0].fill_diagonal_(1.0)
    wd = eye.to(torch.float8_e4m3fn).view(torch.uint8)
    su = torch.full((1, 2, 2), 0.25, device="cuda")
    sd = torch.ones((1, 2, 2), device="cuda")
    value = codes.to(torch.uint8).view(torch.float8_e4m3fn).float() * 0.25
    for base in range(0, 256, 64):
        x = torch.zeros((64, H), device="cuda")
        x[torch.arange(64), base + torch.arange(64)] = 1.0
        ids = torch.zeros((64, 1), dtype=torch.int32, device="cuda")
        y = fp8q.moe_few_tokens(x.bfloat16(), ids, torch.ones((64, 1), device="cuda"), None, None, wu, su, wd, sd,
                                out_dtype=torch.float32)
        assert torch.equal(y, value[base:base + 64, None].expand(64, H))


def test_strided_rows_and_untouched_padding(fp8q):
    ids, share = routing(5, 2, 4)
    w = layer(4, 256, 128)
    x = tokens(5, 256, pad=24)
    want = fp8q.moe_few_tokens(x.contiguous(), ids, share, *w)
    y = torch.full((7, 272), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.randint(0, 256, (fp8q.lib().fp8q_moe_few_tokens_workspace(5, 2, 4, 256, 128),), device="cuda").to(torch.uint8)
    fp8q.fp8q_moe_few_tokens(x, ids, share, *w, y[:5, :256], ws)
    assert torch.equal(y[:5, :256], want) and torch.all(y[5:] == 7.0) and torch.all(y[:, 256:] == 7.0)


def test_no_tokens(fp8q):
    y = fp8q.moe_few_tokens(tokens(0, 256), torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                            torch.empty((0, 2), device="cuda"), *layer(2, 256, 128))
    assert y.shape == (0, 256)


def test_captured_replayed_and_on_two_streams(fp8q):
    """A captured call replayed on new inputs, and two calls at once on two streams, equal the single calls."""
    w = layer(6, 512, 256)
    ids, share = routing(9, 3, 6)
    x = tokens(9, 512)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fp8q.moe_few_tokens(x, ids, share, *w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = fp8q.moe_few_tokens(x, ids, share, *w)
    for seed in (1, 2):
        x.copy_(tokens(9, 512, seed))
        ids.copy_(routing(9, 3, 6, seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, fp8q.moe_few_tokens(x, ids, share, *w))
    xs = [tokens(9, 512, 5), tokens(9, 512, 6)]
    want = [fp8q.moe_few_tokens(v, ids, share, *w) for v in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(fp8q.moe_few_tokens(xs[i], ids, share, *w))
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[i]) for i in (0, 1) for v in got[i])


def test_matches_the_grouped_path(fp8q):
    """Without a gate the layer is the grouped up and down projections plus the weighted sum.  The grouped path
    quantizes x and the hidden rows to E4M3 (relative error 2^-4 each at most, random in sign), the few-token form
    does not: they agree to that in norm (3 % each in the root mean square, 2^-4 / sqrt(3); 6 % together, 10 % allowed)."""
    E, H, I, T = 3, 512, 256, 7
    _, _, wu, su, wd, sd = layer(E, H, I, False)
    ids, share = routing(T, 1, E)
    x = tokens(T, H)
    y = fp8q.moe_few_tokens(x, ids, share, None, None, wu, su, wd, sd, out_dtype=torch.float32)
    rows, pos, off = fp8q.moe_dispatch_layout(ids, E)
    q = torch.empty((T, H), dtype=torch.uint8, device="cuda")
    sf = torch.empty((H // 128, 8), device="cuda")
    fp8q.fp8q_quant_act_1x128_gather(x, rows, q, sf)
    hq = torch.empty((T, I), dtype=torch.uint8, device="cuda")
    hs = torch.empty((I // 128, 8), device="cuda")
    fp8q.fp8q_grouped_gemm_blockscaled_q1x128(q, sf, wu, su, off, hq, hs)
    d = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    fp8q.fp8q_grouped_gemm_blockscaled(hq, hs, wd, sd, off, d)
    long = torch.zeros((T, H), device="cuda")
    long[rows.long()] = d.float()
    long *= share
    assert (long - y).norm() / y.norm() < 0.1
