"""Sizes that the operators' kernels cannot count in 32 bits are refused on the
host, before any CUDA call; the largest that they can count are not."""
import os
import re

import pytest
import torch

import dense_gemm_f32_gb300 as dg

TOP = 2 ** 31 - 1
MAX = 2 ** 31 - 1024


def _p(i):
    return (i + 1) << 44  # fake addresses far apart: never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_f32_gb300 import build

    build.build()


def _ln(rows, cols):
    return dg.dgemm_layer_norm(dg.DTYPE_BF16, rows, cols, 1e-5, _p(0), cols, _p(1), _p(2), _p(3), cols,
                               _p(4), _p(5))


def _ln_bwd(rows, cols):
    return dg.dgemm_layer_norm_backward(dg.DTYPE_F32, rows, cols, _p(0), cols, _p(1), cols, _p(2), _p(3),
                                        _p(4), _p(5), cols, _p(6), cols, _p(7), _p(8))


def _linear(M, N, K):
    return dg.dgemm_linear(dg.DTYPE_F16, 1, 0, M, N, K, _p(0), K, _p(1), N, _p(2), _p(3), N, _p(4), N,
                           _p(5), N)


def _linear_bwd(M, N, K):
    return dg.dgemm_linear_backward(dg.DTYPE_F16, 1, 0, M, N, K, _p(0), N, _p(1), K, _p(2), N, _p(3), N,
                                    _p(4), N, _p(5), K, _p(6), N, _p(7))


def _gated(M, D, F):
    return dg.dgemm_gated_ffn(dg.DTYPE_BF16, 4, 0, M, D, F, _p(0), D, _p(1), F, _p(2), F, _p(3), D, _p(4),
                              D, _p(5), F, _p(6), F, _p(7), F, _p(8), D)


def _gated_bwd(M, D, F):
    lds = (D, D, F, F, D, F, F, F, F, F, D, F, F, D)
    args = [v for i, ld in enumerate(lds) for v in (_p(i), ld)]
    return dg.dgemm_gated_ffn_backward(dg.DTYPE_BF16, 4, 0, M, D, F, *args)


PRODUCTS = (_linear, _linear_bwd, _gated, _gated_bwd)


@pytest.mark.parametrize("size", [MAX + 1, TOP - 254, TOP])
def test_sizes_past_the_limit_are_refused(size):
    for call in PRODUCTS:
        for at in range(3):
            sizes = [1, 1, 1]
            sizes[at] = size
            assert call(*sizes) == dg.ERR_INVALID_VALUE, (call.__name__, sizes)
    for call in (_ln, _ln_bwd):
        assert call(1, size) == dg.ERR_INVALID_VALUE


def test_the_largest_sizes_pass_the_host_checks():
    if torch.cuda.is_available():
        pytest.skip("fake addresses are for machines without a GPU")
    device = (dg.ERR_CUDA, dg.ERR_ARCH)  # what is left to fail
    for call in PRODUCTS:
        for at in range(3):
            sizes = [1, 1, 1]
            sizes[at] = MAX
            assert call(*sizes) in device, (call.__name__, sizes)
    for call in (_ln, _ln_bwd):
        assert call(1, MAX) in device
        assert call(TOP, 1) in device  # rows are counted in 64 bits


def test_the_documented_limit():
    root = os.path.dirname(os.path.dirname(os.path.abspath(dg.__file__)))
    header = open(os.path.join(root, "include", "dgemm.h"), encoding="utf-8").read()
    assert int(re.search(r"DGEMM_OPS_MAX_SIZE (\d+)", header).group(1)) == MAX
