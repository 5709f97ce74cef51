"""The orthogonalised update over spectra from flat to steep, low rank and matrices of few
distinct values, held to the limit that its documentation states (newton_spectra.py), whatever
way the kernels take there."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import newton_reference as nr
import newton_spectra as ns
from ops_reference import U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    gu.check_watchdog()


SIZES = [(64, 128), (200, 100), (256, 512), (512, 576), (512, 1200), (1500, 520), (1024, 2048), (1030, 1024)]


def _off(x, **kw):
    """Distance of the update, in fp32, from the formula in 64 bits; of its norm."""
    got = dg.orthogonalize(x, out=torch.empty(x.shape, device="cuda"), **kw).double()
    assert torch.isfinite(got).all()
    steps, c = kw.get("steps", 5), kw.get("coefficients", nr.MUON)
    want = nr.formula(x.double(), steps, c)
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("rows, cols", SIZES)
@pytest.mark.parametrize("name", ns.NAMES)
def test_within_the_documented_limit(name, rows, cols, dtype):
    assert _off(ns.make(name, rows, cols, dtype).cuda()) <= ns.LIMIT


@pytest.mark.parametrize("steps", [1, 2, 3, 4])
@pytest.mark.parametrize("rows, cols", [(256, 512), (512, 1200), (1030, 1024)])
@pytest.mark.parametrize("name", ns.NAMES)
def test_fewer_steps(name, rows, cols, steps):
    """Each step less enlarges what was rounded by a less."""
    assert _off(ns.make(name, rows, cols, torch.float16).cuda(), steps=steps) <= ns.LIMIT
