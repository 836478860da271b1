"""The rows of layer_mean_rows have the means they claim, and their bounds fail a one-pass variance."""
import pytest
import torch

import layer_mean_rows as D
import layer_reference as R


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [256, 512, 2048, 7168])
def test_bounds_tell_a_one_pass_variance(dtype, N):
    x = D.rows(8, N, dtype, N)
    assert D.ratio(x) > (2000 if dtype == torch.float32 else 500)
    _, _, r, _ = R.layer_norm(x, None, None, D.EPS)
    one = D.one_pass_rstd(x).double()
    assert not ((one - r).abs() <= D.rstd_bound(x) * r).all()
    c = torch.full((2, N), D.CONSTANT[dtype], dtype=dtype)
    assert (c.float() * c.float() != c.double() * c.double()).all() == (dtype == torch.float32)
    _, low, high = D.constant_bounds(c[0, 0].item())
    if dtype == torch.float32:
        one = D.one_pass_rstd(c).double()
        assert not ((one >= low) & (one <= high)).all()
