"""Refusals of the orthogonalised update, none of which needs a GPU, and its reference."""
import ctypes

import pytest
import torch

import dense_gemm_f32_gb300 as dg
import newton_reference as nr

P = 0x10000000  # fake, 16-byte aligned addresses far apart: never dereferenced
BF, HF, F32 = dg.DTYPE_BF16, dg.DTYPE_F16, dg.DTYPE_F32
C = nr.MUON * 5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_f32_gb300 import build

    build.build()


def _call(xt=BF, t=BF, steps=5, c=C, eps=1e-7, scale=1.0, keep=1.0, rows=4, cols=8, X=P, ldx=8, R=2 * P, ldr=8,
          D=3 * P, ldd=8, work=4 * P):
    return dg.dgemm_orthogonalize(xt, t, steps, c, eps, scale, keep, rows, cols, X, ldx, R, ldr, D, ldd, work, 0)


@pytest.mark.parametrize("bad, status", [
    (dict(xt=3), dg.ERR_UNSUPPORTED), (dict(t=-1, rows=-1), dg.ERR_UNSUPPORTED),
    (dict(rows=-1), dg.ERR_INVALID_VALUE), (dict(cols=-1), dg.ERR_INVALID_VALUE),
    (dict(ldx=7), dg.ERR_INVALID_VALUE), (dict(ldr=7), dg.ERR_INVALID_VALUE), (dict(ldd=7), dg.ERR_INVALID_VALUE),
    (dict(steps=0), dg.ERR_INVALID_VALUE), (dict(steps=65, c=[1.0] * 195), dg.ERR_INVALID_VALUE),
    (dict(eps=-1.0), dg.ERR_INVALID_VALUE), (dict(eps=float("nan")), dg.ERR_INVALID_VALUE),
    (dict(eps=float("inf")), dg.ERR_INVALID_VALUE), (dict(scale=float("inf")), dg.ERR_INVALID_VALUE),
    (dict(keep=float("nan")), dg.ERR_INVALID_VALUE), (dict(c=(65.0,) + C[1:]), dg.ERR_INVALID_VALUE),
    (dict(c=C[:14] + (float("nan"),)), dg.ERR_INVALID_VALUE), (dict(cols=2 ** 31 - 1000), dg.ERR_INVALID_VALUE),
    (dict(c=None), dg.ERR_NULL_POINTER), (dict(X=0), dg.ERR_NULL_POINTER), (dict(D=0), dg.ERR_NULL_POINTER),
    (dict(work=0), dg.ERR_NULL_POINTER), (dict(X=P + 1), dg.ERR_MISALIGNED),
    (dict(t=F32, D=3 * P + 2), dg.ERR_MISALIGNED), (dict(work=4 * P + 8), dg.ERR_MISALIGNED),
    (dict(D=P), dg.ERR_ALIAS), (dict(D=2 * P, ldd=9), dg.ERR_ALIAS), (dict(work=P + 16), dg.ERR_ALIAS),
    (dict(D=4 * P + 64), dg.ERR_ALIAS),
])
def test_refusals(bad, status):
    assert _call(**bad) == status


@pytest.mark.parametrize("empty", [dict(rows=0, X=0, D=0), dict(cols=0, ldx=1, ldr=1, ldd=1, work=0)])
def test_nothing_to_write_is_a_no_op(empty):
    assert _call(**empty) == dg.OK


def test_an_update_in_place_is_no_alias():
    assert _call(D=2 * P) in (dg.ERR_CUDA, dg.ERR_ARCH, dg.ERR_INVALID_POINTER)


def test_workspace_holds_two_matrices_and_five_squares():
    for r, c in ((1, 1), (997, 1013), (70000, 3)):
        m = min(r, c)
        assert dg.dgemm_orthogonalize_workspace(r, c) >= 4 * r * ((c + 7) // 8 * 8) + 10 * m * ((m + 7) // 8 * 8)
    assert dg.dgemm_orthogonalize_workspace(0, 4) == 0 and dg.dgemm_orthogonalize_workspace(4, -1) == 0


def test_too_few_coefficients():
    with pytest.raises(ValueError, match="15 coefficients"):
        _call(c=C[:14])
    assert ctypes.sizeof(ctypes.c_float) == 4


def test_tensor_call_checks_shapes_and_types():
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    for args, kw, err in [
        ((x.to(torch.int8),), {}, TypeError), ((x[None],), {}, ValueError), ((x[0],), {}, ValueError),
        ((x.t(),), {}, ValueError), ((x,), dict(steps=0), ValueError), ((x,), dict(steps=65), ValueError),
        ((x,), dict(steps="5"), TypeError), ((x,), dict(coefficients=(1.0, 2.0)), ValueError),
        ((x,), dict(coefficients=[(1.0, 2.0, 3.0)] * 4), ValueError), ((x,), dict(coefficients=3.0), TypeError),
        ((x,), dict(coefficients=[(1.0, 2.0)] * 5), ValueError), ((x,), dict(coefficients=(1.0, "a", 2.0)), TypeError),
        ((x,), dict(coefficients=(1.0, float("inf"), 2.0)), ValueError), ((x,), dict(eps="x"), TypeError),
        ((x,), dict(residual=x[:3]), ValueError), ((x,), dict(residual=x.to(torch.int8)), TypeError),
        ((x,), dict(residual=x, out=x.float()), TypeError), ((x,), dict(out=x[:, :8]), ValueError),
        ((x,), {}, ValueError),  # not on a GPU
    ]:
        with pytest.raises(err):
            dg.orthogonalize(*args, **kw)
    with pytest.raises(RuntimeError, match="orthogonalize does not record gradients"):
        dg.orthogonalize(x.float().requires_grad_())


def test_reference_finds_a_planted_mistake():
    """The bounds of newton_reference.py tell a result with a wrong coefficient, a missing step, or
    products in bfloat16 from the right one."""
    gen = torch.Generator().manual_seed(0)
    x = torch.randn((60, 200), generator=gen)
    right = nr.rounded(x.double()).float()
    nr.check(right, x)
    bf = x.double() / x.double().norm()
    for _ in range(5):
        r = lambda t: t.bfloat16().double()  # noqa: E731
        A = r(bf @ bf.T)
        bf = r(nr.MUON[0] * bf + r(nr.MUON[1] * A + nr.MUON[2] * A @ A) @ bf)
    wrong = [nr.rounded(x.double(), 4), nr.rounded(x.double(), 5, (3.4445, -4.7750, 2.03)), bf,
             nr.rounded(x.double()) * 1.01]
    for w in wrong:
        with pytest.raises(AssertionError):
            nr.check(w.float(), x)
