"""The streaming backward pass of the layer norm launches no more blocks than are resident at once: a row of partial sums a
block, so the workspace tells."""
import pytest
import torch

from common import load_fp8q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8q():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return load_fp8q()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(8192, 520), (8192, 1024), (8192, 2048), (8191, 4096), (1184, 1024)])
def test_blocks_fit_at_once(fp8q, M, N, dtype):
    x = torch.ones((M, N), dtype=dtype, device="cuda")
    mean, rstd = torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")
    dg, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    ws = torch.full((fp8q.lib().fp8q_layer_norm_backward_workspace(M, N),), float("nan"), device="cuda")
    fp8q.fp8q_layer_norm_backward(x, x, None, mean, rstd, dgamma=dg, dbeta=db, workspace=ws)
    rows = ws.view(-1, 2, N)
    written = ~rows.isnan().any(2).any(1)
    blocks = int(written.sum())
    assert written[:blocks].all() and rows[blocks:].isnan().all()
    # three stages of two rows of x and of dy, in at most 228 KB an SM
    assert 0 < blocks <= 148 * (228 * 1024 // (3 * 2 * 2 * N * x.element_size()))
    assert torch.all(dg == M) and torch.all(db == M)
