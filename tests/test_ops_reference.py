"""The 64-bit reference forms' gradients against central differences of their
forward forms (CPU): the formulas the GPU results are held to are right."""
import pytest
import torch

import ops_reference as ref


def _rand(seed):
    gen = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)


def _differences(f, inputs, grads, seed):
    """<grad, v> against (f(x + h v) - f(x - h v)) / 2h for a random direction v of each input."""
    r = _rand(seed)
    h = 1e-5
    for i, (x, g) in enumerate(zip(inputs, grads)):
        v = r(*x.shape)
        args = list(inputs)
        args[i] = x + h * v
        up = f(*args)
        args[i] = x - h * v
        want = (up - f(*args)) / (2 * h)
        got = (g * v).sum()
        assert abs(got - want) <= 1e-6 * (1 + abs(want)), f"input {i}: {got} against {want}"


@pytest.mark.parametrize("name", [a for a in ref.ACTS if a != "relu"])
def test_activation_derivatives(name):
    z = torch.linspace(-6, 6, 401, dtype=torch.float64)
    h = 1e-6
    diff = (ref.act(name, z + h)[0] - ref.act(name, z - h)[0]) / (2 * h)
    assert (diff - ref.act(name, z)[1]).abs().max() < 1e-8


def test_relu_is_zero_and_flat_at_zero():
    z = torch.tensor([-1.0, 0.0, 2.0], dtype=torch.float64)
    value, slope = ref.act("relu", z)
    assert value.tolist() == [0, 0, 2] and slope.tolist() == [0, 0, 1]


@pytest.mark.parametrize("name", ["none", "gelu", "gelu_tanh", "silu"])
def test_linear_gradients(name):
    r = _rand(1)
    x, w, b, c = r(5, 7), r(7, 4), r(4), r(5, 4)
    f = lambda x, w, b: (c * ref.linear(x, w, b, name, None, torch.float32)[0][0]).sum()  # noqa: E731
    z = ref.linear(x, w, b, name, None, torch.float32)[1][0]
    g = [v for v, _ in ref.linear_backward(c, x, w, name, z, torch.float32)]
    _differences(f, (x, w, b), g, 2)


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu"])
def test_gated_gradients(name):
    r = _rand(3)
    x, wg, wu, wd, c = r(5, 6), r(6, 8), r(6, 8), r(8, 6), r(5, 6)
    f = lambda x, a, b, d: (c * ref.gated(x, a, b, d, name, None, torch.float32)[0][0]).sum()  # noqa: E731
    got = ref.gated_backward(c, x, wg, wu, wd, x @ wg, x @ wu, name, torch.float32)
    _differences(f, (x, wg, wu, wd), [v for v, _ in got], 4)


def test_layer_norm_gradients():
    r = _rand(5)
    x, w, b, c, dr = r(4, 9), r(9), r(9), r(4, 9), r(4, 9)
    f = lambda x, w, b: (c * ref.layer_norm(x, w, b, 1e-5, torch.float32)[0][0]).sum() + (dr * x).sum()  # noqa: E731
    (_, _), (mu, _), (rs, _) = ref.layer_norm(x, w, b, 1e-5, torch.float32)
    got = ref.layer_norm_backward(c, x, w, mu, rs, dr, torch.float32)
    _differences(f, (x, w, b), [v for v, _ in got], 6)


def test_a_wrong_value_is_found():
    """The comparison itself: one element moved by more than its bound fails."""
    r = _rand(7)
    x, w = r(8, 16), r(16, 8)
    want = ref.linear(x, w, None, "silu", None, torch.float16)[0]
    good = want[0].to(torch.float16)
    ref.check(good, want, "rounded")
    for at in (0, 37, 63):
        bad = good.clone()
        bad.view(-1)[at] += bad.view(-1)[at].abs() * 0.01 + 0.01
        with pytest.raises(AssertionError):
            ref.check(bad, want, "moved")
