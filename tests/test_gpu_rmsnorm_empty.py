"""Rows of no elements: their mean is that of nothing, and every output is written."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_of_no_elements(dtype, residual):
    import aware_conv_amd as A
    z = lambda *n, d=torch.float32: torch.zeros(*n, dtype=d, device="cuda")  # noqa: E731
    x = z(2, 70, 0, d=dtype)
    res = z(2, 70, 0) if residual else None
    scale = torch.full((2, 70), 7.0, device="cuda")
    q, got, _ = A.rmsnorm_fwd_e4m3(x, z(0), residual=res, scale=scale)
    assert got is scale and (scale == 0).all() and q.shape == x.shape
    torch.full((2, 70), 7.0, device="cuda")  # what the allocator hands out next
    y, total, rstd = A.rmsnorm_fwd(x, z(0), residual=res, save_rstd=True)
    assert y.shape == x.shape and rstd.isnan().all() and (total is None) == (not residual)
