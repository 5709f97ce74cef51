"""Sums of signed bytes that reach 2^24, which the 8-bit products hold exactly on every kernel:
1024 products of -128 by -128, 1040 of 127 by 127."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    gu.check_watchdog()


PLANS = [dict(ROW=1), dict(ROW=0, PAIR=0, SPLITS=1), dict(ROW=0, PAIR=0, SPLITS=4), dict(ROW=0, PAIR=1)]


@pytest.mark.parametrize("plan", PLANS, ids=str)
@pytest.mark.parametrize("K, x_byte, w_byte", [(1024, -128, -128), (1024, -128, 127), (1024, 127, -128),
                                               (1040, 127, 127), (1024, None, None)])
def test_sums_up_to_2_to_24_are_exact(K, x_byte, w_byte, plan, monkeypatch):
    for k, v in plan.items():
        monkeypatch.setenv("DGEMM_INT8_" + k, str(v))
    M, N = (3 if plan["ROW"] else 70), 300
    gen = torch.Generator(device="cuda").manual_seed(K)

    def some(rows, byte):
        if byte is None:
            return torch.randint(-128, 128, (rows, K), generator=gen, dtype=torch.int8, device="cuda")
        return torch.full((rows, K), byte, dtype=torch.int8, device="cuda")

    x, w = some(M, x_byte), some(N, w_byte)
    sums = x.double() @ w.double().T
    assert float(sums.abs().max()) <= 2.0 ** 24
    # scales of powers of two keep the sum's bits; a residual takes the rounded sum away before the result
    # is rounded, which leaves the low ones, all but the last two of 13 whatever they are
    args = dict(x_scale=torch.ones(M, device="cuda"), dtype=torch.float16)
    scale = torch.full((N,), 2.0 ** -16, device="cuda")
    high = (sums * 2.0 ** -16).half()
    assert torch.equal(dg.linear_int8(x, w, scale, **args), high)
    low = sums * 2.0 ** -16 - high.double()
    assert torch.equal(dg.linear_int8(x, w, scale, residual=-high, **args), low.half())
