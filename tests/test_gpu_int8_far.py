"""8-bit products and quantisation past 2^31 elements and bytes: the last rows are those of a call
on the last rows alone (the same bits: a token's and a feature's sums do not depend on
the others, and integers of this size add up exactly in any cut)."""
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


def _int8(rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    return torch.randint(-15, 16, (rows, cols), generator=gen, dtype=torch.int8, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_far_outputs_and_residuals(dtype):
    M, N, K = 33000, 65600, 32
    x, w = torch.randn((M, K), device="cuda").to(dtype), _int8(N, K)
    s = torch.full((N,), 0.01, device="cuda")
    out = torch.full((M, N), 1.0, dtype=dtype, device="cuda")
    got = dg.linear_int8(x, w, s, residual=out, out=out)
    one = torch.ones((70, N), dtype=dtype, device="cuda")
    for rows in (slice(0, 70), slice(16380, 16450), slice(M - 70, M)):
        assert torch.equal(got[rows], dg.linear_int8(x[rows], w, s, residual=one))
    del got, out


@pytest.mark.parametrize("M", [1, 4, 16, 600])
def test_far_weights(M):
    K, N = 65552, 33000
    w, s = _int8(N, K), torch.full((N,), 0.01, device="cuda")
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    got = dg.linear_int8(x, w, s)
    for rows in (slice(0, 100), slice(N - 100, N)):
        want = dg.linear_int8(x, w[rows], s[rows])
        # |q w| sums to about 65552 * 32 * 8 = 2^24: exact
        assert torch.equal(got[:, rows], want)


@pytest.mark.parametrize("transpose", [False, True])
def test_far_rows(transpose):
    M, N = 33000, 65600
    x = torch.randn((M, N), device="cuda", dtype=torch.bfloat16)
    q, s = dg.quantize_int8(x, transpose=transpose)
    for rows in (slice(0, 8), slice(M - 8, M)) if not transpose else (slice(0, 8), slice(N - 8, N)):
        part = x[rows] if not transpose else x[:, rows]
        want, ws = dg.quantize_int8(part.contiguous(), transpose=transpose)
        assert torch.equal(q[rows], want) and torch.equal(s[rows], ws)
