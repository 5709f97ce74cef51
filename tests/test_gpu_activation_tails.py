"""Activations and their derivatives element by element over both tails, relative
to the stored value.

The products only carry the values: with unit matrices for weights every sum has
one term, so an output element is one activation, rounded once.  Tolerances:
  half a unit in the last place of the stored type: at most 2^-8 of a bf16
           value, 2^-11 of an fp16 one (below fp16's normal range 2^-25)
  evaluation in fp32: 2^-15 of the terms' magnitudes.  The exponentials'
           arguments are below 50 on |z| <= 8 and off by a few 2^-24 of
           themselves, which moves a result by up to 150 2^-24; erfc by 2 x^2 =
           64 times its argument's 2^-23; the factors of a derivative (1 - s
           times up to 120 at z = 8) by 120 1.5 2^-23
"""
import math

import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import ops_reference as ref

pytestmark = pytest.mark.gpu
TINY = {torch.bfloat16: 2.0 ** -125, torch.float16: 2.0 ** -25}
EVAL = 2.0 ** -15


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def expected(name, z):
    """act(z), act'(z) and the magnitudes of the terms that act' is the sum of, in 64 bits, in
    forms that do not cancel in the tails."""
    if name == "gelu":
        cdf, rest = 0.5 * torch.erfc(-z / math.sqrt(2)), z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    elif name in ("gelu_tanh", "silu"):
        a, b = (2 * math.sqrt(2 / math.pi), 0.044715) if name == "gelu_tanh" else (1.0, 0.0)
        cdf = torch.sigmoid(a * (z + b * z ** 3))
        rest = z * cdf * (1 - cdf) * a * (1 + 3 * b * z * z)
    else:
        value, slope = ref.act(name, z)
        return value, slope, slope
    return z * cdf, cdf + rest, cdf + rest.abs()


def _close(got, want, magnitude, dtype, z, what):
    bound = ref.U[dtype] * (want.abs() + EVAL * magnitude) + EVAL * magnitude + TINY[dtype]
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()}; first at z = {z[bad][0].item()}: got "
        f"{got[bad][0].item()!r}, want {want[bad][0].item()!r}, bound {bound[bad][0].item()!r}")


def _arguments(dtype):
    """Every fourth value of the type in [-8, 8] above 2^-6 in magnitude, in rows of eight."""
    bits = torch.arange(0, 1 << 15, dtype=torch.int32).to(torch.int16).view(dtype)
    z = bits[(bits.float() <= 8) & (bits.float() > 2.0 ** -6)][::4]
    z = torch.cat([z, -z, torch.zeros(8, dtype=dtype)])
    return z[: z.numel() // 8 * 8].view(-1, 8).cuda()


def check_linear(name, dtype, z, value, slope, terms):
    """act(z) and act'(z) through a linear layer and its backward pass."""
    eye = torch.eye(8, dtype=dtype, device="cuda")
    got = dg.linear(z, eye, activation=name)
    _close(got, value, value.abs(), dtype, z, f"{name}")
    dx, _, _ = dg.linear_backward(torch.ones_like(z), torch.zeros_like(z), eye, activation=name, preact=z)
    _close(dx, slope, terms, dtype, z, f"{name}'")
    gu.check_watchdog()


def check_gated(name, dtype, z, value, slope, terms):
    """u = 1: h = act(g), dg = act'(g), du = act(g)."""
    one, eye = torch.ones_like(z), torch.eye(8, dtype=dtype, device="cuda")
    none = torch.zeros_like(eye)
    x = torch.cat([z, one], 1)
    wg, wu = torch.cat([eye, none]), torch.cat([none, eye])  # g = z, u = 1
    wd = torch.cat([eye, none], 1)                           # y = [h, 0]
    y = dg.gated_ffn(x, wg, wu, wd, activation=name)
    _close(y[:, :8], value, value.abs(), dtype, z, f"{name}")
    dx, _, _, _ = dg.gated_ffn_backward(x.new_ones(x.shape), torch.zeros_like(x), wg, wu, wd, z, one,
                                        activation=name)
    _close(dx[:, :8], slope, terms, dtype, z, f"{name}'")
    _close(dx[:, 8:], value, value.abs(), dtype, z, f"{name} in du")
    gu.check_watchdog()


@pytest.mark.parametrize("pair", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("name", ref.ACTS)
def test_linear(name, dtype, pair, monkeypatch):
    monkeypatch.setenv("DGEMM_FUSED_PAIR", str(pair))
    z = _arguments(dtype)
    check_linear(name, dtype, z, *expected(name, z.double()))


@pytest.mark.parametrize("pair", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("name", ref.ACTS)
def test_gated(name, dtype, pair, monkeypatch):
    monkeypatch.setenv("DGEMM_FUSED_PAIR", str(pair))
    z = _arguments(dtype)
    check_gated(name, dtype, z, *expected(name, z.double()))
