"""The few-token MoE layer's hidden rows keep FP32's accuracy.  One-hot tokens and an identity down projection make
every dot product a single exact term, so that the result shows the hidden value itself.

Bound of an FP32 result, relative, u = 2^-24 half a step of FP32: the up product's scales (the code's product is
exact) 3 u, gated twice that, its silu and product 16 u (expf, sum, quotient, product); the hidden value's 22 bits 2^-22;
the down product's scales 3 u, the weighted sum 1 u; products on the tensor cores add one term and zeros, and at most two
parts: 4 u.  Together under 2^-22 + 33 u < 2^-18.  The hidden value's own part has to show beside it: one FP16 number
(2^-11) fails by two orders."""
import pytest
import torch

import layer_reference as R
from common import load_fp8q

pytestmark = pytest.mark.gpu
REL = 2.0 ** -22 + 33 * R.U


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


def one_hot_layer(E, H, I, gated, seed):
    """Up (and gate) weights of full-mantissa scales, a down projection that copies hidden value i to columns i, I + i, ..."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def weight():
        w = (torch.randn((E, I, H), generator=g, device="cuda") * 112).clamp(-448, 448).to(torch.float8_e4m3fn)
        return w.view(torch.uint8), (torch.rand((E, I // 128, H // 128), generator=g, device="cuda") + 0.5) * 0.02

    wg, sg = weight() if gated else (None, None)
    wu, su = weight()
    eye = torch.eye(I, device="cuda").repeat((H + I - 1) // I, 1)[:H].to(torch.float8_e4m3fn).view(torch.uint8)
    wd = eye[None].repeat(E, 1, 1).contiguous()
    sd = torch.rand((E, H // 128, I // 128), generator=g, device="cuda") + 0.5
    return wg, sg, wu, su, wd, sd


# few, more and many entries (the three sizes of items), whole and partly filled last steps of K
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 1, 2, 256, 128), (5, 3, 4, 384, 1152), (30, 4, 5, 256, 640), (80, 8, 9, 384, 384)])
def test_hidden_values_keep_22_bits(fp8q, T, k, E, H, I, gated):
    g = torch.Generator(device="cuda").manual_seed(T)
    w = one_hot_layer(E, H, I, gated, T + I)
    x = torch.zeros((T, H), device="cuda")
    at = torch.randint(0, H, (T,), generator=g, device="cuda")
    x[torch.arange(T, device="cuda"), at] = torch.randn(T, generator=g, device="cuda") * 0.3
    x = x.bfloat16()
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda").int()
    slot = torch.randint(0, k, (T,), generator=g, device="cuda")
    share = torch.zeros((T, k), device="cuda")
    share[torch.arange(T, device="cuda"), slot] = torch.rand(T, generator=g, device="cuda") + 0.5
    y = fp8q.moe_few_tokens(x, ids, share, *w, out_dtype=torch.float32).double()
    for t in range(T):
        e, c = int(ids[t, slot[t]]), int(at[t])
        col = lambda codes, sf: R.dequant(codes[e], sf[e])[:, c] * x[t, c].double()      # noqa: E731
        h = col(w[2], w[3])
        if gated:
            v = col(w[0], w[1])
            h = v / (1 + torch.exp(-v)) * h
        want = share[t, slot[t]].double() * (R.dequant(w[4][e], w[5][e]) @ h)
        # under 2^-40 of its 128's largest a hidden value is one FP16 step's
        floor = 2.0 ** -38 * (share[t, slot[t]].double() * (R.dequant(w[4][e], w[5][e]).abs() @ torch.full_like(h, h.abs().max())))
        assert ((y[t] - want).abs() <= REL * want.abs() + floor).all(), ((y[t] - want).abs() / want.abs()).max()
    assert fp8q.fp8q_device_status() == 0


def test_bf16_rows_are_the_fp32_rows_rounded(fp8q):
    """One computation for both output types."""
    w = one_hot_layer(3, 512, 256, True, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((11, 512), generator=g, device="cuda").bfloat16()
    ids = torch.randint(0, 3, (11, 2), generator=g, device="cuda").int()
    share = torch.rand((11, 2), generator=g, device="cuda")
    y = fp8q.moe_few_tokens(x, ids, share, *w, out_dtype=torch.float32)
    assert torch.equal(fp8q.moe_few_tokens(x, ids, share, *w), y.bfloat16())
