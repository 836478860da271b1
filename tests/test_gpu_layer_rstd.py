"""A row's rstd comes from its variance by the same correctly rounded root and reciprocal in every kernel: rows of zeros,
whose variance is exactly zero, get the bits of 1 / sqrt(eps) so rounded, whatever the number of rows."""
import numpy as np
import pytest
import torch

from common import load_fp8q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


# a warp a row, a block a row, the streams
@pytest.mark.parametrize("M,N", [(5, 256), (5, 1024), (2400, 1024)])
def test_rstd_of_rows_of_zeros(fp8q, M, N):
    x = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    for i in range(60):
        eps = np.float32(1e-6 * 1.37 ** i)
        want = np.float32(1.0) / np.sqrt(eps)
        _, mean, rstd = fp8q.layer_norm(x, eps=float(eps))
        assert torch.all(mean == 0) and torch.all(rstd == float(want)), (eps, want, rstd[0].item())
