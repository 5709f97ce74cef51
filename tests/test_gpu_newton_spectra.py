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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
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


PLANS = [dict(PAIR=1), dict(PAIR=0, SPLITS=1, TN=64), dict(PAIR=0, SPLITS=1, TN=128), dict(PAIR=0, SPLITS=2),
         dict(PAIR=0, SPLITS=8)]


@pytest.mark.parametrize("plan", PLANS, ids=str)
@pytest.mark.parametrize("rows, cols", [(40, 60), (60, 40), (130, 520), (520, 130), (257, 255), (513, 1030), (700, 515)])
@pytest.mark.parametrize("name", ["rank one", "i^-2", "eight over a floor"])
def test_both_terms_of_fp32_on_every_kernel_and_cut(name, rows, cols, plan, monkeypatch):
    """Where either term of an fp32 matrix were lost, a matrix of rank one would be off by 0.15."""
    for k, v in plan.items():
        monkeypatch.setenv("DGEMM_NEWTON_" + k, str(v))
    x = ns.make(name, rows, cols, torch.float32).cuda()
    assert _off(x) <= ns.LIMIT
    assert _off(x, steps=1) <= 2.0 ** -10  # one group: P of 2^-12, the result stored in fp32
    wide = torch.full((rows, cols + 3), float("nan"), device="cuda")
    wide[:, 1:cols + 1] = x
    assert torch.equal(dg.orthogonalize(wide[:, 1:cols + 1]), dg.orthogonalize(x))


def test_fp32_matrices_that_fp16_holds_are_those():
    """Nothing is left of them for the second term: the result of the fp16 matrix, to the last bit."""
    x = ns.make("i^-1", 300, 700, torch.float16).cuda()
    out = [torch.empty(x.shape, device="cuda") for _ in range(2)]
    assert torch.equal(dg.orthogonalize(x, out=out[0]), dg.orthogonalize(x.float(), out=out[1]))


@pytest.mark.parametrize("dtype, least", [(torch.float32, -149), (torch.bfloat16, -133)], ids=str)
@pytest.mark.parametrize("rows, cols", [(64, 100), (512, 600)])
def test_the_ends_of_the_types(rows, cols, dtype, least):
    """A power of two on X changes nothing where eps is 0, down to subnormal numbers and up to
    the largest ones, whose squares' sum is 2^270."""
    gen = torch.Generator().manual_seed(1)
    x = torch.randint(-7, 8, (rows, cols), generator=gen).double().cuda()
    out = [torch.empty((rows, cols), device="cuda") for _ in range(2)]
    want = dg.orthogonalize(x.to(dtype), eps=0.0, out=out[0])
    assert torch.isfinite(want).all()
    for up in (least, least + 4, least + 20, -100, -60, -30, 30, 60, 100, 120, 125):
        y = (x * 2.0 ** up).to(dtype)
        assert torch.equal(y.double(), x * 2.0 ** up)
        assert torch.equal(dg.orthogonalize(y, eps=0.0, out=out[1]), want), up


GENTLE = {"cubic": ((1.5, -0.5, 0.0), 6), "quintic": ((15 / 8, -10 / 8, 3 / 8), 6)}


@pytest.mark.parametrize("plan", PLANS, ids=str)
@pytest.mark.parametrize("c, steps", GENTLE.values(), ids=GENTLE.keys())
@pytest.mark.parametrize("rows, cols", [(130, 520), (520, 130), (513, 1030), (1030, 1024)])
@pytest.mark.parametrize("name", ["flat", "i^-1", "i^-3", "rank one", "two values, 1.7"])
def test_longer_groups_of_gentle_steps(name, rows, cols, c, steps, plan, monkeypatch):
    """Three and four steps among m x m matrices, the next Gram matrix and the product of the
    polynomials in one launch: a growth of 2^4 as with two steps of the usual coefficients, and the
    steps after the group enlarge what it rounds by a^3 = 6.6 at most, not 40.9, so by less than
    the limit."""
    for k, v in plan.items():
        monkeypatch.setenv("DGEMM_NEWTON_" + k, str(v))
    for dtype in (torch.float16, torch.float32):
        x = ns.make(name, rows, cols, dtype).cuda()
        assert _off(x, steps=steps, coefficients=c) <= ns.LIMIT


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("m", [2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("n", [1, 8, 100, 1400])
def test_few_rows_or_columns(m, n, dtype):
    """Products of two vectors with some noise, whose second singular value is small."""
    gen = torch.Generator().manual_seed(m)
    for noise in (0.03, 0.1, 0.3, 1.0):
        for _ in range(6):
            x = torch.randn((m, 1), generator=gen) * torch.randn((1, m + n), generator=gen)
            x = (x + noise * torch.randn(x.shape, generator=gen)).to(dtype).cuda()
            assert _off(x) <= ns.FEW and _off(x.t().contiguous()) <= ns.FEW
