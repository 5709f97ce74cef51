"""The backward layer norm's ring when a copy never comes and many rows are
still to be copied: the call comes back, the status names the site, and what
runs next on the same SMs is right."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import ops_reference as ref
from test_gpu_fused_watchdog import _stalled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    gu.check_watchdog()


# 8 to 100 rows per group of threads, rings of 8 down to 2 stages
@pytest.mark.parametrize("rows, cols, dtype", [
    (rows, cols, dtype) for dtype in (torch.bfloat16, torch.float32)
    for rows, cols in ((40000, 300), (16000, 1000), (6000, 4096), (1500, 8192))] + [(1500, 8200, torch.float16)])
def test_a_ring_that_gave_up_is_refilled_no_more(rows, cols, dtype, monkeypatch):
    n = ref.make(6)
    x, dy = n((rows, cols), dtype), n((rows, cols), dtype)
    dr = n((rows, cols), dtype)
    _, mean, rstd = dg.layer_norm(x, return_stats=True)
    call = lambda: dg.layer_norm_backward(dy, x, None, mean, rstd, dresidual=dr)  # noqa: E731
    _stalled(call, "norm.cu", monkeypatch)
    one = torch.ones(cols, dtype=torch.float64, device="cuda")
    want = ref.layer_norm_backward(dy.double(), x.double(), one, mean.double(), rstd.double(), dr.double(),
                                   dtype)
    for g, w_, what in zip(call(), want, ("dx", "dweight", "dbias")):
        ref.check(g, w_, what)
