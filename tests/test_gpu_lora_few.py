"""Adapters for about a token a group: groups of none, one, two and more tokens, ranks on both sides of the short rows,
odd widths, against the 64-bit formula within layer_reference's bound."""
import pytest
import torch

from common import load_fp8q
from test_gpu_lora import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,n,r,K,N", [(1, 1, 8, 64, 8), (1, 1, 16, 64, 72), (5, 6, 16, 520, 264), (40, 64, 8, 128, 1032),
                                       (33, 33, 16, 264, 2056), (33, 33, 24, 264, 2056), (65, 64, 16, 1024, 18432),
                                       (66, 64, 16, 256, 4104), (500, 600, 16, 136, 520), (500, 600, 8, 136, 40)])
def test_about_a_token_a_group(fp8q, T, n, r, K, N, dtype):
    x, a, b, scaling, base, ids = make(T, n, r, K, N, dtype, seed=T + n + r)
    check(fp8q, x, ids, a, b, scaling, base)
    check(fp8q, x, ids, a, b, None, base)


@pytest.mark.parametrize("r", [8, 16])
def test_all_tokens_in_one_group(fp8q, r):
    x, a, b, scaling, base, ids = make(31, 40, r, 256, 1048, "bf16", seed=r, pad=8)
    ids.fill_(17)
    check(fp8q, x, ids, a, b, scaling, base)
    ids[:15] = 40                                  # no adapter
    check(fp8q, x, ids, a, b, scaling, base)
