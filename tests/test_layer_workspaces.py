"""The workspaces of the operators around a projection, on the host: a start that the kernels' vector accesses cannot use
is refused; and the norm's partial rows are no more than its steps need."""
import pytest

from common import load_fp8q

FAKE = 1 << 20        # fake device address (never dereferenced)


@pytest.fixture(scope="module")
def fp8q():
    return load_fp8q()


# row kernels, a warp and a block a row; the streams, which store their partial rows two floats at a time
@pytest.mark.parametrize("M,N", [(100, 256), (100, 1000), (1184, 520), (8192, 7168)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_norm_backward_workspace_alignment(fp8q, M, N, dtype):
    L = fp8q.lib()
    need = L.fp8q_layer_norm_backward_workspace(M, N)

    def call(ws, dgamma, dbeta):
        return L.fp8q_layer_norm_backward(FAKE, N, FAKE, N, dtype, M, N, FAKE, 1, FAKE, FAKE, FAKE, N, dgamma, dbeta, ws,
                                          need, None)

    for offset in (4, 8, 12):
        for dgamma, dbeta in ((FAKE, FAKE), (FAKE, None), (None, FAKE)):
            assert call(FAKE + offset, dgamma, dbeta) == fp8q.FP8Q_ERR_ALIGNMENT
    # no device here, or a launch on one: what is left to refuse is not the workspace's start
    if not fp8q.torch.cuda.is_available():
        assert call(FAKE, FAKE, FAKE) == fp8q.FP8Q_ERR_CUDA
        assert call(FAKE + 4, None, None) == fp8q.FP8Q_ERR_CUDA          # no weight gradients: it is not used


@pytest.mark.parametrize("M", [1184, 1185, 2368, 5000, 8192])
@pytest.mark.parametrize("N", [520, 1024, 1536, 2048, 3584])
def test_partial_rows_of_the_streams(fp8q, M, N):
    """A block of the streams, and so a partial row, has at least as many steps of two rows as its ring has stages."""
    rows = fp8q.lib().fp8q_layer_norm_backward_workspace(M, N) // (2 * N)
    assert rows <= ((M + 1) // 2 + 2) // 3
