"""Bounded waits of the 8-bit products' kernels that run out: the call comes
back, the status names a site of the kernel, and the next call is right."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import int8_reference as ref8
import ops_reference as ref
from test_gpu_fused_watchdog import _stalled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    gu.check_watchdog()


def _plan(monkeypatch, plan):
    for k, v in plan.items():
        monkeypatch.setenv("DGEMM_INT8_" + k, str(v))


PLANS = [dict(ROW=0, PAIR=0, SPLITS=1), dict(ROW=0, PAIR=0, SPLITS=4), dict(ROW=0, PAIR=1, NT=64),
         dict(ROW=0, PAIR=1, NT=192)]


@pytest.mark.parametrize("plan", PLANS, ids=str)
@pytest.mark.parametrize("K", [48, 1024, 5008])
def test_linear_wait_runs_out(plan, K, monkeypatch):
    _plan(monkeypatch, plan)
    n = ref.make(K)
    x, w = n((500, K), torch.float16), dg.quantize_int8(n((520, K), torch.float16, K ** -0.5))
    call = lambda: dg.linear_int8(x, *w, activation="relu")  # noqa: E731
    want = call()
    ref.check(want, ref8.linear(*ref8.quantize(x), w[0].double(), w[1].double(), None, "relu", None, torch.float16),
              "before")
    _stalled(call, "int8_pair.cu" if plan["PAIR"] else "int8_small.cu", monkeypatch)
    assert torch.equal(call(), want)


@pytest.mark.parametrize("plan", [PLANS[0], PLANS[3]], ids=str)
def test_block_wait_runs_out(plan, monkeypatch):
    _plan(monkeypatch, plan)
    n = ref.make(9)
    x = n((300, 512), torch.bfloat16)
    weights = [t for s in ((640, 512), (640, 512), (512, 640)) for t in dg.quantize_int8(n(s, torch.bfloat16, 0.05))]
    call = lambda: dg.gated_ffn_int8(x, *weights)  # noqa: E731
    want = call()
    _stalled(call, "int8_pair.cu" if plan["PAIR"] else "int8_small.cu", monkeypatch)
    assert torch.equal(call(), want)
