"""The documented limit of an orthogonalised update's error tells what it should, on the CPU: with
the roundings of newton_reference.py, groups of steps of the size that the library takes stay within
it and longer first groups do not, nor does an fp32 matrix that is rounded to fp16 first."""
import pytest
import torch

import newton_reference as nr
import newton_spectra as ns


def _update(x, groups, terms=1):
    """Five steps in groups, m x m matrices and the iterate rounded to fp16; X in one or two terms."""
    up = 2.0 ** (8 - torch.floor(torch.log2(x.norm())) - 1)
    hi = (x * up).half().double()
    lo = (x * up - hi).half().double() if terms == 2 else 0.0
    x = (hi + lo) / (x.norm() * up)
    eye, (a, b, c) = torch.eye(x.shape[0], dtype=x.dtype), nr.MUON
    for g, steps in enumerate(groups):
        A, Q = nr._stored(x @ x.T), None
        for i in range(steps):
            P = nr._stored(a * eye + b * A + c * A @ A)
            Q = P if Q is None else nr._stored(Q @ P)
            if i + 1 < steps:
                A = nr._stored(nr._stored(A @ P) @ P)
        x = Q @ x
        if g + 1 < len(groups):
            x = nr._half(x, 256.0)
    return x


def _off(name, rows, cols, dtype, groups, terms=1):
    x = ns.make(name, rows, cols, dtype).double()
    want = nr.formula(x)
    return float((_update(x, groups, terms) - want).norm() / want.norm())


@pytest.mark.parametrize("rows, cols, groups", [(64, 128, (2, 1, 1, 1)), (512, 576, (2, 1, 1, 1)),
                                                (512, 900, (2, 1, 2))])
@pytest.mark.parametrize("name", ns.NAMES)
def test_the_groups_taken_stay_within_the_limit(name, rows, cols, groups):
    assert _off(name, rows, cols, torch.float16, groups) <= ns.LIMIT
    assert _off(name, rows, cols, torch.float32, groups, terms=2) <= ns.LIMIT


@pytest.mark.parametrize("name", ["rank one", "two values, 1.7", "equal rows"])
def test_three_steps_at_first_do_not(name):
    assert _off(name, 512, 576, torch.float16, (3, 2)) > 1.2 * ns.LIMIT


@pytest.mark.parametrize("name", ["rank one", "i^-3", "rank three"])
def test_an_fp32_matrix_in_one_term_does_not(name):
    assert _off(name, 64, 128, torch.float32, (2, 1, 1, 1), terms=1) > 1.2 * ns.LIMIT
