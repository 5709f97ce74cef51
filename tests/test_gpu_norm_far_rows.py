"""Layer norm backward of rows so far from zero that what pads a row in the
kernel must not be normalised with it."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("cols", [5, 8, 40, 264, 1000, 4104])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_far_rows_do_not_meet_their_padding(dtype, cols):
    """x = mean = 1e36, rstd = 1e4: (x - mean) rstd is 0 in every column, but (0 - mean) rstd is
    past fp32's range.  dx = rstd (p - mean(p)) stays finite."""
    n = ref.make(cols)
    x = torch.full((4, cols), 1e36, device="cuda").to(dtype)
    dy = n((4, cols), dtype, 0.1)
    w = n((cols,), dtype, 0.2, 1.0)
    mean, rstd = x[:, 0].float().contiguous(), torch.full((4,), 1e4, device="cuda")
    got = dg.layer_norm_backward(dy, x, w, mean, rstd)
    p = dy.double() * w.double()
    c = (cols / 32 + 40) * 2.0 ** -24
    want = 1e4 * (p - p.mean(1, keepdim=True))
    bound = 1e4 * c * (p.abs() + p.abs().mean(1, keepdim=True))
    ref.check(got[0], (want, bound * (1 + ref.U[dtype]) + ref.stored(want, dtype)), "dx")
    assert not got[1].any()  # xh = 0
    db = dy.double().sum(0)
    ref.check(got[2], (db, 12 * ref.E * dy.double().abs().sum(0) + ref.stored(db, dtype)), "dbias")
    gu.check_watchdog()
