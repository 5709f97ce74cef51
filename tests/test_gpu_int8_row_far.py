"""The 8-bit products' kernel for few tokens (csrc/int8_row.cu) with weights past 2^31 bytes and
with the longest rows that it takes, on aligned rows and on others: the formula on the first and
the last features, to the last bit (32-bit sums are exact; two products in fp32 and one
rounding follow)."""
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


@pytest.mark.parametrize("off", [0, 5], ids=["aligned", "odd rows"])
@pytest.mark.parametrize("M, K, N", [(1, 65536, 33000), (1, 65521, 33000), (2, 65536, 33000), (4, 40000, 54000),
                                     (3, 40929, 53000)])
def test_far_and_long_rows_of_weights(M, K, N, off, monkeypatch):
    monkeypatch.setenv("DGEMM_INT8_ROW", "1")
    gen = torch.Generator(device="cuda").manual_seed(K)
    pitch = (K + 15) // 16 * 16 + off
    store = torch.randint(-128, 128, (off + N * pitch,), generator=gen, dtype=torch.int8, device="cuda")
    w = store.as_strided((N, K), (pitch, 1), off)
    assert w.data_ptr() + (N - 1) * pitch - store.data_ptr() > 2 ** 31
    ws = torch.rand((N,), generator=gen, device="cuda") * 1e-3
    x = torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16)
    q, s = dg.quantize_int8(x)
    launches = dg.dgemm_kernel_launches()
    got = dg.linear_int8(x, w, ws)
    assert dg.dgemm_kernel_launches() == launches + 1  # the one kernel, which quantises the tokens itself
    given = dg.linear_int8(q, w, ws, x_scale=s)
    assert torch.equal(given, got)
    for rows in (slice(0, 40), slice(N // 2, N // 2 + 40), slice(N - 40, N)):
        sums = (q.double() @ w[rows].double().T).float()
        assert torch.equal(got[:, rows], (sums * ws[rows] * s[:, None]).to(torch.bfloat16))
