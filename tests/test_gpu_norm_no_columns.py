"""Layer norm of rows without columns."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_rows_without_columns_have_no_statistics(dtype):
    """The mean of nothing is not a number, and never what the memory held before."""
    for n in (1, 6, 300):
        for _ in range(2):  # what the statistics' memory held before
            torch.full((n,), 7.0, device="cuda")
        x = torch.empty((n, 0), dtype=dtype, device="cuda")
        y, mean, rstd = dg.layer_norm(x, x.new_empty(0), x.new_empty(0), return_stats=True)
        assert y.shape == (n, 0) and mean.shape == rstd.shape == (n,)
        assert torch.isnan(mean).all() and torch.isnan(rstd).all()
        dx, dw, db = dg.layer_norm_backward(y, x, None, mean, rstd)
        assert dx.shape == (n, 0) and dw.shape == db.shape == (0,)
