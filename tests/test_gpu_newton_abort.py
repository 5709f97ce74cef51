"""Bounded waits of the update's kernels that run out, on the CTA pairs with inputs of the epilogue in
flight and where a cluster joins parts of K: the call comes back, the status names a site of
the kernel, and the next call is right."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import newton_reference as nr
import ops_reference as ref
from test_gpu_fused_watchdog import _stalled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    gu.check_watchdog()


PLANS = [dict(PAIR=1), dict(PAIR=0, SPLITS=4), dict(PAIR=0, SPLITS=8), dict(PAIR=0, SPLITS=1, TN=128)]


@pytest.mark.parametrize("plan", PLANS, ids=str)
@pytest.mark.parametrize("rows, cols, x_type, w_type", [(600, 900, torch.bfloat16, torch.bfloat16),
                                                        (900, 601, torch.float32, torch.float32)], ids=str)
def test_update_with_a_residual_wait_runs_out(rows, cols, x_type, w_type, plan, monkeypatch):
    for k, v in plan.items():
        monkeypatch.setenv("DGEMM_NEWTON_" + k, str(v))
    n = ref.make(rows)
    x, w = n((rows, cols), x_type), n((rows, cols), w_type, 0.05)
    args = dict(steps=1, scale=-0.02, residual=w, residual_scale=0.9)
    want = dg.orthogonalize(x, **args)
    nr.check(want, x, 1, scale=-0.02, residual=w, keep=0.9)
    _stalled(lambda: dg.orthogonalize(x, **args), "newton_pair.cu" if plan["PAIR"] else "newton_small.cu",
             monkeypatch)
    assert torch.equal(dg.orthogonalize(x, **args), want)
