"""Activations and their derivatives of finite arguments whose square or cube is
past fp32's range: their limits, act(z) = max(z, 0) and act'(z) = 0 or 1."""
import pytest
import torch

import gpu_util as gu
import ops_reference as ref
from test_gpu_activation_tails import check_gated, check_linear

pytestmark = pytest.mark.gpu
# 1e20 squared is past fp32's range; fp16 ends at 65504
HUGE = {torch.bfloat16: (1e4, 1e12, 1e20, 3e38), torch.float16: (1e3, 3e4, 6e4, 65504.0)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def _inputs(dtype, sign):
    return (sign * torch.tensor(HUGE[dtype] * 2, dtype=dtype))[None].cuda()


def _limits(name, z):
    value, slope = (z, torch.ones_like(z)) if name == "none" else (z.clamp(min=0), (z > 0).double())
    return value, slope, slope


@pytest.mark.parametrize("pair", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("sign", [1, -1])
def test_huge_arguments(sign, name, dtype, pair, monkeypatch):
    monkeypatch.setenv("DGEMM_FUSED_PAIR", str(pair))
    z = _inputs(dtype, sign)
    check_linear(name, dtype, z, *_limits(name, z.double()))
    check_gated(name, dtype, z, *_limits(name, z.double()))
    gu.check_watchdog()
