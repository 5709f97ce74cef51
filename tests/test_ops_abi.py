"""Refusals of the feed-forward operators, none of which needs a GPU: the C
entry points check on the host before any CUDA call, in the documented order,
and the tensor calls check shapes and types first."""
import os
import re

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


def _ln(dtype=BF, rows=4, cols=8, eps=1e-5, X=_p(0), ldx=8, w=_p(1), b=_p(2), Y=_p(3), ldy=8,
        mean=_p(4), rstd=_p(5)):
    return dg.dgemm_layer_norm(dtype, rows, cols, eps, X, ldx, w, b, Y, ldy, mean, rstd, 0)


def _ln_bwd(dtype=BF, rows=4, cols=8, dY=_p(0), lddy=8, X=_p(1), ldx=8, w=_p(2), mean=_p(3),
            rstd=_p(4), dR=_p(5), lddr=8, dX=_p(6), lddx=8, dw=_p(7), db=_p(8)):
    return dg.dgemm_layer_norm_backward(dtype, rows, cols, dY, lddy, X, ldx, w, mean, rstd, dR,
                                        lddr, dX, lddx, dw, db, 0)


def _linear(dtype=BF, act=1, op=0, M=4, N=8, K=16, X=_p(0), ldx=16, W=_p(1), ldw=8, b=_p(2),
            R=_p(3), ldr=8, D=_p(4), ldd=8, Z=_p(5), ldz=8):
    return dg.dgemm_linear(dtype, act, op, M, N, K, X, ldx, W, ldw, b, R, ldr, D, ldd, Z, ldz, 0)


def _linear_bwd(dtype=BF, act=1, op=0, M=4, N=8, K=16, dD=_p(0), lddd=8, X=_p(1), ldx=16, W=_p(2),
                ldw=8, Z=_p(3), ldz=8, dZ=_p(4), lddz=8, dX=_p(5), lddx=16, dW=_p(6), lddw=8,
                db=_p(7)):
    return dg.dgemm_linear_backward(dtype, act, op, M, N, K, dD, lddd, X, ldx, W, ldw, Z, ldz, dZ,
                                    lddz, dX, lddx, dW, lddw, db, 0)


def _gated(dtype=BF, act=4, op=0, M=4, D=8, F=16, X=_p(0), ldx=8, Wg=_p(1), ldwg=16, Wu=_p(2),
           ldwu=16, Wd=_p(3), ldwd=8, R=_p(4), ldr=8, H=_p(5), ldh=16, G=_p(6), ldg=16, U=_p(7),
           ldu=16, Y=_p(8), ldy=8):
    return dg.dgemm_gated_ffn(dtype, act, op, M, D, F, X, ldx, Wg, ldwg, Wu, ldwu, Wd, ldwd, R, ldr,
                              H, ldh, G, ldg, U, ldu, Y, ldy, 0)


def _gated_bwd(dtype=BF, act=4, op=0, M=4, D=8, F=16, **kw):
    names = [("dY", D), ("X", D), ("Wg", F), ("Wu", F), ("Wd", D), ("G", F), ("U", F), ("H", F),
             ("dG", F), ("dU", F), ("dX", D), ("dWg", F), ("dWu", F), ("dWd", D)]
    args = []
    for i, (n, ld) in enumerate(names):
        args += [kw.pop(n, _p(i)), kw.pop("ld" + n.lower(), max(ld, 1))]
    assert not kw
    return dg.dgemm_gated_ffn_backward(dtype, act, op, M, D, F, *args, 0)


CALLS = {"layer_norm": _ln, "layer_norm_backward": _ln_bwd, "linear": _linear,
         "linear_backward": _linear_bwd, "gated_ffn": _gated, "gated_ffn_backward": _gated_bwd}
PRODUCTS = [c for c in CALLS if "norm" not in c]


@pytest.mark.parametrize("name", CALLS)
def test_unknown_type_activation_or_layout_comes_first(name):
    call = CALLS[name]
    assert call(dtype=3) == dg.ERR_UNSUPPORTED
    assert call(dtype=-1) == dg.ERR_UNSUPPORTED
    size = "rows" if "norm" in name else "M"
    assert call(dtype=9, **{size: -1}) == dg.ERR_UNSUPPORTED
    if name in PRODUCTS:
        assert call(dtype=F32) == dg.ERR_UNSUPPORTED  # the products take 16-bit operands
        assert call(act=5) == dg.ERR_UNSUPPORTED
        assert call(act=-1) == dg.ERR_UNSUPPORTED
        assert call(op=2) == dg.ERR_UNSUPPORTED


@pytest.mark.parametrize("name, bad", [
    ("layer_norm", dict(rows=-1)), ("layer_norm", dict(cols=-1)), ("layer_norm", dict(ldx=7)),
    ("layer_norm", dict(ldy=7)), ("layer_norm", dict(eps=-1e-5)),
    ("layer_norm", dict(eps=float("nan"))), ("layer_norm", dict(eps=float("inf"))),
    ("layer_norm_backward", dict(lddy=7)), ("layer_norm_backward", dict(ldx=7)),
    ("layer_norm_backward", dict(lddr=7)), ("layer_norm_backward", dict(lddx=7)),
    ("linear", dict(M=-1)), ("linear", dict(N=-1)), ("linear", dict(K=-1)),
    ("linear", dict(ldx=15)), ("linear", dict(ldw=7)), ("linear", dict(op=1, ldw=15)),
    ("linear", dict(ldr=7)), ("linear", dict(ldd=7)), ("linear", dict(ldz=7)),
    ("linear_backward", dict(lddd=7)), ("linear_backward", dict(ldz=7)),
    ("linear_backward", dict(lddz=7)), ("linear_backward", dict(lddx=15)),
    ("linear_backward", dict(lddw=7)), ("linear_backward", dict(op=1, ldw=16, lddw=15)),
    ("gated_ffn", dict(F=-1)), ("gated_ffn", dict(ldwg=15)), ("gated_ffn", dict(ldwu=15)),
    ("gated_ffn", dict(ldwd=7)), ("gated_ffn", dict(ldh=15)), ("gated_ffn", dict(ldg=15)),
    ("gated_ffn", dict(ldy=7)),
    ("gated_ffn_backward", dict(D=-1)), ("gated_ffn_backward", dict(lddy=7)),
    ("gated_ffn_backward", dict(lddg=15)), ("gated_ffn_backward", dict(lddwd=7)),
])
def test_bad_sizes_are_refused(name, bad):
    assert CALLS[name](**bad) == dg.ERR_INVALID_VALUE


@pytest.mark.parametrize("name, empty", [
    ("layer_norm", dict(rows=0)), ("layer_norm", dict(cols=0, ldx=1, ldy=1)),
    ("layer_norm_backward", dict(rows=0, dw=0, db=0)), ("linear", dict(M=0)),
    ("linear", dict(N=0, X=0, W=0, D=0)), ("linear_backward", dict(dX=0, dW=0, db=0)),
    ("linear_backward", dict(M=0, dW=0, db=0)), ("gated_ffn", dict(M=0, X=0, Y=0)),
    ("gated_ffn", dict(D=0, F=0)), ("gated_ffn_backward", dict(D=0)),
    ("gated_ffn_backward", dict(dX=0, dWg=0, dWu=0, dWd=0)),
])
def test_nothing_to_write_is_a_no_op(name, empty):
    assert CALLS[name](**empty) == dg.OK


@pytest.mark.parametrize("name, missing", [
    ("layer_norm", "X"), ("layer_norm", "Y"), ("layer_norm_backward", "dY"),
    ("layer_norm_backward", "X"), ("layer_norm_backward", "mean"), ("layer_norm_backward", "rstd"),
    ("layer_norm_backward", "dX"), ("linear", "X"), ("linear", "W"), ("linear", "D"),
    ("linear_backward", "dD"), ("linear_backward", "X"), ("linear_backward", "W"),
    ("linear_backward", "Z"), ("linear_backward", "dZ"), ("gated_ffn", "X"), ("gated_ffn", "Wg"),
    ("gated_ffn", "Wu"), ("gated_ffn", "Wd"), ("gated_ffn", "H"), ("gated_ffn", "Y"),
    ("gated_ffn", "G"), ("gated_ffn", "U"), ("gated_ffn_backward", "dY"),
    ("gated_ffn_backward", "G"), ("gated_ffn_backward", "H"), ("gated_ffn_backward", "dWg"),
    ("gated_ffn_backward", "dWu"),
])
def test_missing_matrices_are_refused(name, missing):
    assert CALLS[name](**{missing: 0}) == dg.ERR_NULL_POINTER


@pytest.mark.parametrize("name, odd", [
    ("layer_norm", dict(X=_p(0) + 1)), ("layer_norm", dict(dtype=F32, X=_p(0) + 2)),
    ("layer_norm", dict(mean=_p(4) + 2)), ("layer_norm_backward", dict(rstd=_p(4) + 2)),
    ("linear", dict(W=_p(1) + 1)), ("linear", dict(b=_p(2) + 1)), ("linear", dict(D=_p(4) + 1)),
    ("linear_backward", dict(db=_p(7) + 1)), ("gated_ffn", dict(U=_p(7) + 1)),
    ("gated_ffn_backward", dict(dWd=_p(13) + 1)),
])
def test_misaligned_pointers_are_refused(name, odd):
    assert CALLS[name](**odd) == dg.ERR_MISALIGNED


@pytest.mark.parametrize("name, same", [
    ("layer_norm", dict(Y=_p(0) + 16)), ("layer_norm", dict(Y=_p(0))),
    ("layer_norm", dict(mean=_p(1) + 4)), ("layer_norm_backward", dict(dX=_p(0) + 32)),
    ("layer_norm_backward", dict(dX=_p(5))), ("layer_norm_backward", dict(db=_p(7) + 2)),
    ("linear", dict(D=_p(0))), ("linear", dict(D=_p(3) + 2)), ("linear", dict(D=_p(3), ldd=16)),
    ("linear", dict(Z=_p(4))), ("linear", dict(Z=_p(3))),
    ("linear_backward", dict(dZ=_p(0))), ("linear_backward", dict(dX=_p(4))),
    ("gated_ffn", dict(H=_p(0))), ("gated_ffn", dict(U=_p(6))), ("gated_ffn", dict(Y=_p(0))),
    ("gated_ffn_backward", dict(dU=_p(8))), ("gated_ffn_backward", dict(H=_p(5))),
])
def test_overlapping_outputs_are_refused(name, same):
    assert CALLS[name](**same) == dg.ERR_ALIAS


@pytest.mark.parametrize("name, fine", [
    ("linear", dict(D=_p(3))), ("gated_ffn", dict(Y=_p(4))), ("linear", dict(b=0, R=0, Z=0)),
    ("linear_backward", dict(act=0, Z=0, dZ=0)), ("layer_norm", dict(w=0, b=0, mean=0, rstd=0)),
])
def test_in_place_residual_and_absent_options_pass_the_host_checks(name, fine):
    """Past every check that needs no GPU: what is left is the device."""
    if torch.cuda.is_available():
        pytest.skip("fake addresses are for machines without a GPU")
    assert CALLS[name](**fine) in (dg.ERR_CUDA, dg.ERR_ARCH)


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: dg.linear(_z(2, 3, dtype=torch.float32), _z(3, 4)),
    lambda: dg.linear(_z(2, 3), _z(3, 4, dtype=torch.float16)),
    lambda: dg.linear(_z(2, 3), _z(3, 4), bias=_z(4, dtype=torch.float32)),
    lambda: dg.layer_norm(_z(2, 3, dtype=torch.float64)),
    lambda: dg.layer_norm(_z(2, 3), weight=_z(3, dtype=torch.float32)),
    lambda: dg.gated_ffn(_z(2, 4, dtype=torch.float32), _z(4, 8), _z(4, 8), _z(8, 4)),
    lambda: dg.gated_ffn_backward(_z(2, 4), _z(2, 4), _z(4, 8), _z(4, 8), _z(8, 4),
                                  _z(2, 8, dtype=torch.float16), _z(2, 8)),
])
def test_tensor_calls_refuse_other_types(call):
    with pytest.raises(TypeError):
        call()


@pytest.mark.parametrize("call", [
    lambda: dg.linear(_z(2, 3), _z(4, 3)),
    lambda: dg.linear(_z(2, 3), _z(3, 4), trans_w=True),
    lambda: dg.linear(_z(2, 3), _z(3, 4), bias=_z(3)),
    lambda: dg.linear(_z(2, 3), _z(3, 4), residual=_z(2, 3)),
    lambda: dg.linear(_z(2, 3), _z(3, 4), residual=_z(1, 4)),  # no broadcasting
    lambda: dg.linear(_z(2, 3), _z(3, 4), activation="tanh"),
    lambda: dg.linear(_z(3, 2).t(), _z(3, 4)),
    lambda: dg.linear(_z(2, 3), _z(3, 4), out=_z(2, 3)),
    lambda: dg.linear(_z(2, 6, 3)[:, ::2].transpose(0, 1), _z(3, 4)),
    lambda: dg.linear_backward(_z(2, 4), _z(2, 3), _z(3, 4), activation="silu"),
    lambda: dg.linear_backward(_z(2, 3), _z(2, 3), _z(3, 4)),
    lambda: dg.layer_norm(_z(2, 3), weight=_z(2)),
    lambda: dg.layer_norm(_z(2, 3), bias=_z(1, 3)),
    lambda: dg.layer_norm_backward(_z(2, 4), _z(2, 3), None, torch.zeros(2), torch.zeros(2)),
    lambda: dg.layer_norm_backward(_z(2, 3), _z(2, 3), None, torch.zeros(3), torch.zeros(2)),
    lambda: dg.gated_ffn(_z(2, 4), _z(4, 8), _z(4, 7), _z(8, 4)),
    lambda: dg.gated_ffn(_z(2, 4), _z(4, 8), _z(4, 8), _z(4, 8)),
    lambda: dg.gated_ffn(_z(2, 4), _z(4, 8), _z(4, 8), _z(8, 4), residual=_z(2, 8)),
    lambda: dg.gated_ffn_backward(_z(2, 4), _z(2, 4), _z(4, 8), _z(4, 8), _z(8, 4), _z(2, 8), _z(2, 4)),
])
def test_tensor_calls_refuse_other_shapes(call):
    with pytest.raises(ValueError):
        call()


def test_watchdog_site_codes_are_distinct():
    """Every bounded wait of every kernel has its own site code, across files."""
    root = os.path.join(os.path.dirname(os.path.abspath(dg.__file__)), "csrc")
    codes = []
    for f in sorted(os.listdir(root)):
        text = open(os.path.join(root, f), encoding="utf-8").read()
        codes += re.findall(r"kSite\w+ = (0x[0-9a-f]+)", text)
    assert len(codes) == len(set(codes)) >= 20
