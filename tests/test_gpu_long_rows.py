"""Rows longer than 2^30 elements: byte offsets within a row past 32 bits, on
rows that start on any alignment, read and written by either kernel of the
fused products and by the activation gradient."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu

pytestmark = pytest.mark.gpu
N = (1 << 30) + 129


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


def _row(offset, seed):
    """A 1 x N row of small integers and halves (their sums and products are exact), `offset`
    elements into its buffer."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.empty(offset + N + 64, dtype=torch.float16, device="cuda")
    buf.random_(-8, 8, generator=gen).mul_(0.5)
    return buf, buf[offset:offset + N].view(1, N)


@pytest.mark.parametrize("pair", [0, 1])
@pytest.mark.parametrize("offset", [0, 1])
def test_linear(offset, pair, monkeypatch):
    monkeypatch.setenv("DGEMM_FUSED_PAIR", str(pair))
    (_, w), (_, r), (_, b), (guard, out) = (_row(offset, i) for i in range(4))
    before = guard.clone()
    x = torch.full((1, 1), 3.0, dtype=torch.float16, device="cuda")
    dg.linear(x, w, b[0], residual=r, out=out)
    want = w * 3
    want += b
    want += r
    assert torch.equal(out, want)
    for around in (slice(0, offset), slice(offset + N, None)):  # stays as it was
        assert torch.equal(guard[around], before[around])
    gu.check_watchdog()


@pytest.mark.parametrize("offset", [0, 1])
def test_linear_backward(offset):
    (_, w), (_, z), (_, dd) = (_row(offset, i) for i in range(3))
    x = torch.full((1, 1), 3.0, dtype=torch.float16, device="cuda")
    _, dw, db = dg.linear_backward(dd, x, w, "relu", z)
    dz = dd * (z > 0)
    assert torch.equal(db, dz[0])
    assert torch.equal(dw, dz.mul_(3))
    gu.check_watchdog()
