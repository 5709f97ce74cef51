"""Layer norm of constant rows of 16-bit values whose sum is exact in fp32: the
mean is the value itself, the variance 0 and y the bias, at any number of columns."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


@pytest.mark.parametrize("cols", [3, 7, 100, 333, 997, 1013, 1500, 2047, 4095, 5000, 8191, 8200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
def test_constant_rows(dtype, cols):
    value = torch.tensor([1000.0, -0.337, 7.0, 0.0, 21.3, -3000.0, 1.0 / 3, 49.0]).to(dtype)
    n = ref.make(cols)
    w, b = n((cols,), dtype, 0.2, 1.0), n((cols,), dtype)
    x = value.cuda()[:, None].expand(-1, cols).contiguous()
    y, mean, rstd = dg.layer_norm(x, w, b, eps=1e-5, return_stats=True)
    assert torch.equal(mean, value.float().cuda())
    assert ((rstd.double() * 1e-5 ** 0.5 - 1).abs() < 1e-6).all()
    assert torch.equal(y, b.expand_as(y))
