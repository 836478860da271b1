"""The operators around an FP8 projection, on the host: refusals of the C entry
points and of the binding before anything is launched, and the 64-bit formulas
of layer_reference against central differences."""
import pytest
import torch

import layer_reference as R
from common import load_fp8q

FAKE = 1 << 20        # 16-byte aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def fp8q():
    return load_fp8q()


def test_layer_norm_validation(fp8q):
    L = fp8q.lib()
    INV, ALN, UNS = fp8q.FP8Q_ERR_INVALID_ARG, fp8q.FP8Q_ERR_ALIGNMENT, fp8q.FP8Q_ERR_UNSUPPORTED

    def ln(x=FAKE, dt=0, M=4, N=256, ldx=256, gamma=FAKE, beta=FAKE, pt=1, eps=1e-5, y=FAKE, ldy=256, mean=FAKE,
           rstd=FAKE, q=None, ldq=256, sf=None, ld_sf=4):
        return L.fp8q_layer_norm(x, dt, M, N, ldx, gamma, beta, pt, eps, y, ldy, mean, rstd, q, ldq, sf, ld_sf, None)

    assert ln(dt=2) == INV and ln(pt=-1) == INV and ln(M=-1) == INV and ln(N=0) == INV and ln(ldx=248) == INV
    assert ln(eps=0.0) == INV and ln(eps=-1.0) == INV and ln(eps=float("nan")) == INV and ln(eps=float("inf")) == INV
    assert ln(ldy=248) == INV and ln(x=None) == INV
    assert ln(y=None) == INV                                     # no output
    assert ln(q=FAKE) == INV and ln(sf=FAKE) == INV              # one of the pair
    assert ln(q=FAKE, sf=FAKE, ldq=128) == INV and ln(q=FAKE, sf=FAKE, ld_sf=3) == INV
    assert ln(q=FAKE, sf=FAKE, N=200) == INV                     # N % 128
    assert ln(N=16385, ldx=16392, ldy=16392) == UNS
    assert ln(x=FAKE + 8) == ALN and ln(y=FAKE + 2) == ALN and ln(gamma=FAKE + 4) == ALN and ln(beta=FAKE + 8) == ALN
    assert ln(ldx=260) == ALN and ln(ldy=257) == ALN and ln(dt=1, ldx=258) == ALN
    assert ln(mean=FAKE + 2) == ALN and ln(rstd=FAKE + 1) == ALN
    assert ln(q=FAKE + 8, sf=FAKE) == ALN and ln(q=FAKE, sf=FAKE + 2) == ALN and ln(q=FAKE, sf=FAKE, ldq=264) == ALN
    assert ln(M=0, x=None, y=None) == 0                          # empty: nothing launched


def test_layer_norm_backward_validation(fp8q):
    L = fp8q.lib()
    INV, ALN, UNS = fp8q.FP8Q_ERR_INVALID_ARG, fp8q.FP8Q_ERR_ALIGNMENT, fp8q.FP8Q_ERR_UNSUPPORTED
    need = L.fp8q_layer_norm_backward_workspace(100, 1000)
    assert need == 50 * 2 * 1000                                 # one partial row of each gradient a row pair
    assert L.fp8q_layer_norm_backward_workspace(0, 1000) == 0 and L.fp8q_layer_norm_backward_workspace(4, 16385) == 0

    def lb(dy=FAKE, lddy=1000, x=FAKE, ldx=1000, dt=0, M=100, N=1000, gamma=FAKE, pt=1, mean=FAKE, rstd=FAKE, dx=FAKE,
           lddx=1000, dgamma=FAKE, dbeta=FAKE, ws=FAKE, n=need):
        return L.fp8q_layer_norm_backward(dy, lddy, x, ldx, dt, M, N, gamma, pt, mean, rstd, dx, lddx, dgamma, dbeta,
                                          ws, n, None)

    assert lb(dt=5) == INV and lb(pt=9) == INV and lb(M=-1) == INV and lb(N=0) == INV
    assert lb(lddy=992) == INV and lb(ldx=992) == INV and lb(lddx=992) == INV
    assert lb(dy=None) == INV and lb(x=None) == INV and lb(mean=None) == INV and lb(rstd=None) == INV
    assert lb(dx=None, dgamma=None, dbeta=None) == INV
    assert lb(ws=None) == INV and lb(n=need - 1) == INV and lb(dgamma=None, n=0) == INV
    assert lb(N=16392, lddy=16392, ldx=16392, lddx=16392) == UNS
    assert lb(dy=FAKE + 8) == ALN and lb(x=FAKE + 2) == ALN and lb(dx=FAKE + 4) == ALN and lb(gamma=FAKE + 8) == ALN
    assert lb(ldx=1004) == ALN and lb(lddy=1001) == ALN and lb(lddx=1001) == ALN and lb(dt=1, ldx=1002) == ALN
    assert lb(mean=FAKE + 1) == ALN and lb(dgamma=FAKE + 2) == ALN and lb(dbeta=FAKE + 2) == ALN and lb(ws=FAKE + 2) == ALN


def test_layer_norm_binding_refusals(fp8q):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fp8q.layer_norm(x)                                       # a CPU tensor never reaches the library
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        fp8q._dtype(torch.zeros(4, dtype=torch.float16))
    with pytest.raises(ValueError, match="gamma"):
        fp8q.fp8q_layer_norm(x, torch.ones(255), None, 1e-5, x)
    with pytest.raises(ValueError, match="beta"):                # one parameter type
        fp8q.fp8q_layer_norm(x, torch.ones(256), torch.ones(256, dtype=torch.bfloat16), 1e-5, x)
    with pytest.raises(ValueError, match="y:"):
        fp8q.fp8q_layer_norm(x, None, None, 1e-5, torch.zeros((4, 255), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="sf"):
        fp8q.fp8q_layer_norm(x, None, None, 1e-5, None, q=x.view(torch.uint8)[:, :256], sf=torch.zeros((1, 4)))
    with pytest.raises(ValueError, match="mean"):
        fp8q.fp8q_layer_norm_backward(x, x, None, torch.zeros(3), torch.zeros(4), x)
    with pytest.raises(ValueError, match="dy"):
        fp8q.fp8q_layer_norm_backward(x.float(), x, None, torch.zeros(4), torch.zeros(4), x)


def test_layer_norm_gradient_against_differences():
    """The backward formula equals central differences of the forward formula (64 bits, h = 1e-5: the differences'
    own error is h^2 times a third derivative plus 2^-53 / h, below 1e-8 of the terms)."""
    g = torch.Generator().manual_seed(0)
    M, N, eps, h = 3, 5, 1e-3, 1e-5
    x, dy = torch.randn((M, N), generator=g).double(), torch.randn((M, N), generator=g).double()
    gamma, beta = torch.randn(N, generator=g).double(), torch.randn(N, generator=g).double()
    loss = lambda x, ga, be: (R.layer_norm(x, ga, be, eps)[0] * dy).sum()  # noqa: E731
    _, mean, rstd, _ = R.layer_norm(x, gamma, beta, eps)
    dx, dgamma, dbeta = R.layer_norm_backward(dy, x, gamma, mean, rstd)

    def difference(t, i, f):
        d = torch.zeros_like(t)
        d.view(-1)[i] = h
        return (f(t + d) - f(t - d)) / (2 * h)

    for i in range(M * N):
        assert abs(difference(x, i, lambda t: loss(t, gamma, beta)) - dx.view(-1)[i]) < 1e-7 * (1 + dx.abs().max())
    for i in range(N):
        assert abs(difference(gamma, i, lambda t: loss(x, t, beta)) - dgamma[i]) < 1e-7 * (1 + dgamma.abs().max())
        assert abs(difference(beta, i, lambda t: loss(x, gamma, t)) - dbeta[i]) < 1e-7 * (1 + dbeta.abs().max())


def test_moe_few_tokens_validation(fp8q):
    L = fp8q.lib()
    INV, ALN, UNS = fp8q.FP8Q_ERR_INVALID_ARG, fp8q.FP8Q_ERR_ALIGNMENT, fp8q.FP8Q_ERR_UNSUPPORTED
    size = L.fp8q_moe_few_tokens_workspace
    need = size(4, 2, 8, 256, 128)
    assert need > 0 and size(0, 2, 8, 256, 128) == 0 and size(4, 2, 8, 200, 128) == 0 and size(129, 1, 8, 256, 128) == 0
    # the hidden rows in FP32 and FP16, every entry's output row: at least these
    assert need >= 8 * 128 * 6 + 8 * 256 * 4 + 4 * 256 * 2

    def mf(x=FAKE, T=4, H=256, ldx=256, ids=FAKE, share=FAKE, k=2, E=8, wg=FAKE, sg=FAKE, wu=FAKE, su=FAKE, wd=FAKE,
           sd=FAKE, I=128, y=FAKE, ldy=256, dt=0, ws=FAKE, n=need):
        return L.fp8q_moe_few_tokens(x, T, H, ldx, ids, share, k, E, wg, sg, wu, su, wd, sd, I, y, ldy, dt, ws, n, None)

    assert mf(T=-1) == INV and mf(k=0) == INV and mf(E=0) == INV and mf(H=200, ldx=256) == INV and mf(I=64) == INV
    assert mf(H=0) == INV and mf(I=0) == INV and mf(ldx=248) == INV and mf(ldy=248) == INV and mf(dt=3) == INV
    assert mf(wg=None) == INV and mf(sg=None) == INV                       # one of the pair
    for name in ("x", "ids", "share", "wu", "su", "wd", "sd", "y", "ws"):
        assert mf(**{name: None}) == INV
    assert mf(n=need - 1) == INV
    assert mf(T=129) == UNS and mf(k=257) == UNS and mf(E=1025) == UNS and mf(I=65664) == UNS
    assert mf(H=65664, ldx=65664, ldy=65664) == UNS and mf(k=1 << 40) == INV
    for name in ("x", "wg", "wu", "wd", "y"):
        assert mf(**{name: FAKE + 8}) == ALN
    for name in ("ids", "share", "sg", "su", "sd"):
        assert mf(**{name: FAKE + 2}) == ALN
    assert mf(ws=FAKE + 128) == ALN and mf(ldx=260) == ALN and mf(ldy=260) == ALN and mf(dt=1, ldy=258) == ALN
    assert mf(T=0, x=None, ws=None, n=0) == 0


def test_moe_few_tokens_binding_refusals(fp8q):
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    ids, share = torch.zeros((2, 1), dtype=torch.int32), torch.zeros((2, 1))
    w, sf = torch.zeros((3, 128, 256), dtype=torch.uint8), torch.zeros((3, 1, 2))
    wd, sd = torch.zeros((3, 256, 128), dtype=torch.uint8), torch.zeros((3, 2, 1))
    call = fp8q.moe_few_tokens
    with pytest.raises(ValueError, match="CUDA"):
        call(x, ids, share, w, sf, w, sf, wd, sd)
    with pytest.raises(ValueError, match="expert_ids"):
        call(x, ids.long(), share, w, sf, w, sf, wd, sd)
    with pytest.raises(ValueError, match="x:"):
        call(x.float(), ids, share, w, sf, w, sf, wd, sd)
    with pytest.raises(ValueError, match="w_down"):
        call(x, ids, share, w, sf, w, sf, wd.transpose(1, 2), sd)
    with pytest.raises(ValueError, match="sf_up"):
        call(x, ids, share, w, sf, w, sf[:, :, :1], wd, sd)
    with pytest.raises(ValueError, match="w_gate"):
        call(x, ids, share, w[:2], sf, w, sf, wd, sd)


def test_lora_validation(fp8q):
    L = fp8q.lib()
    INV, ALN, UNS = fp8q.FP8Q_ERR_INVALID_ARG, fp8q.FP8Q_ERR_ALIGNMENT, fp8q.FP8Q_ERR_UNSUPPORTED
    size = L.fp8q_lora_apply_workspace
    need = size(40, 256, 16, 3)
    assert need >= 40 * 16 and size(0, 256, 16, 3) == 0 and size(40, 255, 16, 3) == 0 and size(40, 256, 136, 3) == 0
    assert size(40, 256, 16, 1025) == 0
    # few blocks: the K slices' partial sums lie side by side
    assert size(1, 7168, 16, 1) % 16 == 0 and size(1, 7168, 16, 1) > 16 and size(4096, 7168, 64, 1) == 4096 * 64

    def lo(x=FAKE, T=40, K=256, ldx=256, rows=FAKE, off=FAKE, groups=3, a=FAKE, b=FAKE, r=16, s=FAKE, n=2, base=FAKE,
           ldb=512, out=2 * FAKE, ldo=512, dt=0, N=512, ws=FAKE, wl=need):
        return L.fp8q_lora_apply(x, T, K, ldx, rows, off, groups, a, b, r, s, n, base, ldb, out, ldo, dt, N, ws, wl, None)

    assert lo(T=-1) == INV and lo(K=252) == INV and lo(K=0) == INV and lo(N=508) == INV and lo(r=12) == INV
    assert lo(r=0) == INV and lo(ldx=248) == INV and lo(ldb=504) == INV and lo(ldo=504) == INV
    assert lo(groups=0) == INV and lo(n=-1) == INV and lo(dt=2) == INV
    for name in ("x", "rows", "off", "a", "b", "base", "out", "ws"):
        assert lo(**{name: None}) == INV
    assert lo(wl=need - 1) == INV and lo(out=FAKE, ldo=520) == INV       # in place needs the same rows
    assert lo(r=136) == UNS and lo(groups=1025) == UNS and lo(T=(1 << 24) + 1) == UNS
    for name in ("x", "a", "b", "base", "ws"):
        assert lo(**{name: FAKE + 8}) == ALN
    for name in ("rows", "off", "s"):
        assert lo(**{name: FAKE + 2}) == ALN
    assert lo(out=2 * FAKE + 8) == ALN and lo(ldx=260) == ALN and lo(ldb=516) == ALN and lo(ldo=516) == ALN
    assert lo(dt=1, ldb=514) == ALN
    assert lo(T=0, x=None, out=None, ws=None, wl=0) == 0


def test_lora_binding_refusals(fp8q):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    a, b = torch.zeros((2, 16, 64), dtype=torch.bfloat16), torch.zeros((2, 32, 16), dtype=torch.bfloat16)
    rows, off = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    base = torch.zeros((4, 32), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fp8q.lora_apply(x, rows, off, a, b, None, base)
    with pytest.raises(ValueError, match="rows"):
        fp8q.lora_apply(x, rows.long(), off, a, b, None, base)
    with pytest.raises(ValueError, match="a:"):
        fp8q.lora_apply(x, rows, off, a.float(), b, None, base)
    with pytest.raises(ValueError, match="b:"):
        fp8q.lora_apply(x, rows, off, a, b[:, :, :8], None, base)
    with pytest.raises(ValueError, match="scaling"):
        fp8q.lora_apply(x, rows, off, a, b, torch.ones(3), base)
    with pytest.raises(ValueError, match="base"):
        fp8q.lora_apply(x, rows, off, a, b, None, base[:, :24])
    with pytest.raises(ValueError, match="out"):
        fp8q.lora_apply(x, rows, off, a, b, None, base, out=base.float())
