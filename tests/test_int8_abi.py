"""Refusals of the 8-bit integer products, none of which needs a GPU."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg

P = 0x10000000  # fake, 16-byte aligned addresses far apart: never dereferenced
BF, HF, F32 = dg.DTYPE_BF16, dg.DTYPE_F16, dg.DTYPE_F32


def _p(i):
    return P * (i + 1)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_f32_gb300 import build

    build.build()


def _quant(dtype=BF, op=0, rows=4, cols=8, X=_p(0), ldx=8, Q=_p(1), ldq=8, scale=_p(2)):
    return dg.dgemm_quantize_int8(dtype, op, rows, cols, X, ldx, Q, ldq, scale, 0)


def _linear(dtype=BF, act=1, M=4, N=8, K=16, X=_p(0), ldx=16, xs=0, W=_p(1), ldw=16, ws=_p(2), b=_p(3),
            R=_p(4), ldr=8, D=_p(5), ldd=8, work=_p(6)):
    return dg.dgemm_linear_int8(dtype, act, M, N, K, X, ldx, xs, W, ldw, ws, b, R, ldr, D, ldd, work, 0)


def _gated(dtype=BF, act=4, M=4, D=8, F=16, X=_p(0), ldx=8, Wg=_p(1), ldwg=8, sg=_p(2), Wu=_p(3), ldwu=8,
           su=_p(4), Wd=_p(5), ldwd=16, sd=_p(6), R=_p(7), ldr=8, Y=_p(8), ldy=8, work=_p(9)):
    return dg.dgemm_gated_ffn_int8(dtype, act, M, D, F, X, ldx, Wg, ldwg, sg, Wu, ldwu, su, Wd, ldwd, sd,
                                   R, ldr, Y, ldy, work, 0)


@pytest.mark.parametrize("call, bad, status", [
    (_quant, dict(dtype=3, rows=-1), dg.ERR_UNSUPPORTED), (_quant, dict(op=2), dg.ERR_UNSUPPORTED),
    (_quant, dict(rows=-1), dg.ERR_INVALID_VALUE), (_quant, dict(ldx=7), dg.ERR_INVALID_VALUE),
    (_quant, dict(ldq=7), dg.ERR_INVALID_VALUE), (_quant, dict(op=1, ldq=3), dg.ERR_INVALID_VALUE),
    (_quant, dict(X=0), dg.ERR_NULL_POINTER), (_quant, dict(scale=0), dg.ERR_NULL_POINTER),
    (_quant, dict(Q=0), dg.ERR_NULL_POINTER), (_quant, dict(X=_p(0) + 1), dg.ERR_MISALIGNED),
    (_quant, dict(scale=_p(2) + 2), dg.ERR_MISALIGNED), (_quant, dict(Q=_p(0) + 3), dg.ERR_ALIAS),
    (_quant, dict(rows=2 ** 31 - 1000), dg.ERR_INVALID_VALUE),
    (_linear, dict(dtype=F32), dg.ERR_UNSUPPORTED), (_linear, dict(act=5), dg.ERR_UNSUPPORTED),
    (_linear, dict(M=-1), dg.ERR_INVALID_VALUE), (_linear, dict(ldx=15), dg.ERR_INVALID_VALUE),
    (_linear, dict(ldw=15), dg.ERR_INVALID_VALUE), (_linear, dict(ldr=7), dg.ERR_INVALID_VALUE),
    (_linear, dict(ldd=7), dg.ERR_INVALID_VALUE), (_linear, dict(K=2 ** 31 - 1000), dg.ERR_INVALID_VALUE),
    (_linear, dict(X=0), dg.ERR_NULL_POINTER), (_linear, dict(W=0), dg.ERR_NULL_POINTER),
    (_linear, dict(ws=0), dg.ERR_NULL_POINTER), (_linear, dict(D=0), dg.ERR_NULL_POINTER),
    (_linear, dict(work=0), dg.ERR_NULL_POINTER), (_linear, dict(X=_p(0) + 1), dg.ERR_MISALIGNED),
    (_linear, dict(ws=_p(2) + 2), dg.ERR_MISALIGNED), (_linear, dict(work=_p(6) + 8), dg.ERR_MISALIGNED),
    (_linear, dict(xs=_p(7) + 1), dg.ERR_MISALIGNED), (_linear, dict(D=_p(1)), dg.ERR_ALIAS),
    (_linear, dict(D=_p(4), ldd=9), dg.ERR_ALIAS), (_linear, dict(work=_p(0) + 16), dg.ERR_ALIAS),
    (_linear, dict(D=_p(6) + 128), dg.ERR_ALIAS),
    (_gated, dict(dtype=F32), dg.ERR_UNSUPPORTED), (_gated, dict(act=-1), dg.ERR_UNSUPPORTED),
    (_gated, dict(F=-1), dg.ERR_INVALID_VALUE), (_gated, dict(ldwg=7), dg.ERR_INVALID_VALUE),
    (_gated, dict(ldwd=15), dg.ERR_INVALID_VALUE), (_gated, dict(su=0), dg.ERR_NULL_POINTER),
    (_gated, dict(Wd=0), dg.ERR_NULL_POINTER), (_gated, dict(work=0), dg.ERR_NULL_POINTER),
    (_gated, dict(work=_p(9) + 4), dg.ERR_MISALIGNED), (_gated, dict(Y=_p(0)), dg.ERR_ALIAS),
    (_gated, dict(work=_p(5)), dg.ERR_ALIAS),
])
def test_refusals(call, bad, status):
    assert call(**bad) == status


@pytest.mark.parametrize("call, empty", [
    (_quant, dict(rows=0, X=0)), (_quant, dict(op=1, cols=0, ldx=1, ldq=4)), (_linear, dict(M=0, X=0, work=0)),
    (_linear, dict(N=0, W=0, D=0)), (_gated, dict(M=0)), (_gated, dict(D=0, X=0)),
])
def test_nothing_to_write_is_a_no_op(call, empty):
    assert call(**empty) == dg.OK


def test_odd_byte_addresses_are_fine_and_the_next_check_answers():
    # 8-bit matrices have no alignment: the device is what is missing here
    st = _linear(X=_p(0) + 1, xs=_p(7), W=_p(1) + 3)
    assert st in (dg.ERR_CUDA, dg.ERR_ARCH, dg.ERR_INVALID_POINTER)


def test_workspaces_hold_their_parts():
    for M, K in ((1, 1), (3, 997), (70000, 40000)):
        assert dg.dgemm_linear_int8_workspace(M, K) >= 2 * M * ((K + 7) // 8 * 8) + 4 * M
        assert dg.dgemm_gated_ffn_int8_workspace(M, K, 50) >= 2 * M * ((K + 7) // 8 * 8) + 4 * M * 56 + 4 * M
    assert dg.dgemm_linear_int8_workspace(0, 8) == 0 and dg.dgemm_gated_ffn_int8_workspace(-1, 8, 8) == 0


def _w(n, k):
    return torch.zeros((n, k), dtype=torch.int8), torch.ones(n)


def test_tensor_calls_check_shapes_and_types():
    x, (w, s) = torch.zeros((4, 16), dtype=torch.bfloat16), _w(8, 16)
    xs = torch.ones(4)
    for args, kw, err in [
        ((x.float(), w, s), {}, TypeError), ((x, w.float(), s), {}, TypeError), ((x, w, s.double()), {}, TypeError),
        ((x, w[:, :15], s), {}, ValueError), ((x, w, s[:7]), {}, ValueError), ((x, w.t(), s), {}, ValueError),
        ((x, w, s), dict(x_scale=xs), TypeError), ((x.to(torch.int8), w, s), {}, TypeError),
        ((x.to(torch.int8), w, s), dict(x_scale=xs[:3]), ValueError),
        ((x.to(torch.int8), w, s), dict(x_scale=xs, dtype=torch.float32), TypeError),
        ((x, w, s), dict(dtype=torch.float16), TypeError), ((x, w, s), dict(dtype="bf16"), TypeError),
        ((x, w, s), dict(bias=torch.zeros(8)), TypeError), ((x, w, s), dict(residual=x), ValueError),
        ((x, w, s), dict(out=torch.zeros((4, 8))), TypeError), ((x, w, s), dict(activation="tanh"), ValueError),
        ((x, w, s), {}, ValueError),  # not on a GPU
    ]:
        with pytest.raises(err):
            dg.linear_int8(*args, **kw)
    (wg, sg), (wd, sd) = _w(24, 16), _w(16, 24)
    for bad in ((x.float(), wg, sg, wg, sg, wd, sd), (x, wg, sg, wg[:, :8], sg, wd, sd),
                (x, wg, sg, wg, sg, wd.t(), sd), (x, wg, sg, wg, sg[:3], wd, sd), (x, wg, sg, wg, sg, wd, sd)):
        with pytest.raises((TypeError, ValueError)):
            dg.gated_ffn_int8(*bad)
    for bad in ((x.to(torch.int8),), (x,), (x[None], True)):
        with pytest.raises((TypeError, ValueError)):
            dg.quantize_int8(*bad)


def test_arguments_that_require_gradients_are_refused():
    x, (w, s) = torch.zeros((4, 16), dtype=torch.bfloat16, requires_grad=True), _w(8, 16)
    with pytest.raises(RuntimeError, match="linear_int8 does not record gradients"):
        dg.linear_int8(x, w, s)
    with pytest.raises(RuntimeError, match="does not record"):
        dg.quantize_int8(x)
    with torch.no_grad(), pytest.raises(ValueError):  # past that check: not on a GPU
        dg.quantize_int8(x)
