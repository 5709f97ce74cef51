"""The small kernel when a wait runs out after all its copies have been sent for
(no more stages of K than the ring holds), and in the middle of them."""
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


@pytest.mark.parametrize("splits", [1, 3, 8])
@pytest.mark.parametrize("K", [40, 300, 5000])
def test_copies_in_flight_are_waited_for(K, splits, monkeypatch):
    monkeypatch.setenv("DGEMM_FUSED_PAIR", "0")
    monkeypatch.setenv("DGEMM_FUSED_SPLITS", str(splits))
    n = ref.make(K)
    x, w = n((40, K), torch.float16), n((K, 200), torch.float16, K ** -0.5)
    call = lambda: dg.linear(x, w, activation="relu")  # noqa: E731
    want = call()
    ref.check(want, ref.linear(x.double(), w.double(), None, "relu", None, torch.float16)[0], "before")
    _stalled(call, "fused_small.cu", monkeypatch)
    assert torch.equal(call(), want)
