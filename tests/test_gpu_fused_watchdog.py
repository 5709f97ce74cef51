"""Bounded waits of the operators' kernels that run out: the call comes back,
the status names a site of the kernel, and the next call is right.  (The way of
test_gpu_watchdog.py: one thread waits on a barrier that nothing arrives at, or
a copy is never begun; no fault, no trap, no hang.)"""
import os
import re
import time

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
    yield
    gu.check_watchdog()


def _sites(name):
    path = os.path.join(os.path.dirname(os.path.abspath(dg.__file__)), "csrc", name)
    return {int(c, 16) for c in re.findall(r"kSite\w+ = (0x[0-9a-f]+)", open(path, encoding="utf-8").read())}


def _stalled(call, source, monkeypatch):
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    assert dg.dgemm_watchdog_status(stream)[0] == dg.OK
    monkeypatch.setenv("DGEMM_TC_TEST_STALL", "1")
    t0 = time.time()
    call()
    torch.cuda.synchronize()
    elapsed = time.time() - t0
    monkeypatch.delenv("DGEMM_TC_TEST_STALL")
    st, where = dg.dgemm_watchdog_status(stream)
    assert st == dg.ERR_WATCHDOG and where in _sites(source), (st, hex(where))
    assert elapsed < 30, f"the abort path took {elapsed:.1f} s"
    assert dg.dgemm_watchdog_status(stream)[0] == dg.OK


@pytest.mark.parametrize("plan", [dict(PAIR=1), dict(PAIR=0, SPLITS=1), dict(PAIR=0, SPLITS=4)], ids=str)
def test_linear_wait_runs_out(plan, monkeypatch):
    for k, v in plan.items():
        monkeypatch.setenv("DGEMM_FUSED_" + k, str(v))
    n = ref.make(5)
    x, w = n((600, 1024), torch.bfloat16), n((1024, 520), torch.bfloat16, 0.03)
    call = lambda: dg.linear(x, w, activation="silu")  # noqa: E731
    _stalled(call, "fused_pair.cu" if plan["PAIR"] else "fused_small.cu", monkeypatch)
    ref.check(call(), ref.linear(x.double(), w.double(), None, "silu", None, torch.bfloat16)[0], "after")


@pytest.mark.parametrize("rows, cols", [(500, 300), (400, 2000), (200, 8000)])
def test_layer_norm_backward_wait_runs_out(rows, cols, monkeypatch):
    n = ref.make(6)
    x, dy = n((rows, cols), torch.float16), n((rows, cols), torch.float16)
    _, mean, rstd = dg.layer_norm(x, return_stats=True)
    call = lambda: dg.layer_norm_backward(dy, x, None, mean, rstd)  # noqa: E731
    _stalled(call, "norm.cu", monkeypatch)
    one = torch.ones(cols, dtype=torch.float64, device="cuda")
    want = ref.layer_norm_backward(dy.double(), x.double(), one, mean.double(), rstd.double(), None,
                                   torch.float16)
    for g, w_, what in zip(call(), want, ("dx", "dweight", "dbias")):
        ref.check(g, w_, what)
