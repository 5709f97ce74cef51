"""The tensor calls record nothing for autograd, and say so instead of returning
results that a backward pass would silently stop at."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dense_gemm_f32_gb300 import build

    build.build()


def _z(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _layer_norm():
    return dg.layer_norm, [_z(2, 4), _z(4), _z(4)], {}


def _linear():
    return dg.linear, [_z(2, 4), _z(4, 8), _z(8)], {"residual": _z(2, 8)}


def _gated_ffn():
    return dg.gated_ffn, [_z(2, 4), _z(4, 8), _z(4, 8), _z(8, 4)], {"residual": _z(2, 4)}


@pytest.mark.parametrize("make", [_layer_norm, _linear, _gated_ffn])
def test_arguments_that_require_gradients_are_refused(make):
    call, args, kw = make()
    for at in [*range(len(args)), *kw]:
        call, args, kw = make()
        (kw if isinstance(at, str) else args)[at].requires_grad_()
        with pytest.raises(RuntimeError, match="no_grad"):
            call(*args, **kw)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # past that check
            call(*args, **kw)
        with torch.inference_mode(), pytest.raises(ValueError, match="CUDA"):
            call(*args, **kw)


def test_gradients_are_asked_for_in_any_mode():
    """The backward calls are first-order gradients by themselves."""
    x, w = _z(2, 4), _z(4, 8).requires_grad_()
    with pytest.raises(ValueError, match="CUDA"):
        dg.linear_backward(_z(2, 8), x, w)
