"""64-bit forms of the orthogonalised update, and what its result is held to.

The formula, step by step, is `formula`.  `rounded` is the same result with the
roundings to fp16 that the operator documents (X once per group of steps, every m x m
matrix when it is stored) and nothing else.  Its distance from the formula is
what those roundings give on this input; what is left of the kernels' own
arithmetic, fp32 sums of K terms, is below 2^-24 (K / 16 + 16) of the sums of sizes
per product, a hundredth of a rounding to fp16 at the sizes here, and can only
move the values next to a border of two fp16 numbers.  So a result may be 1.3
times as far from the formula as `rounded` is, in norm, and an element ten times
the root mean square of that, plus the rounding of storing it.  Where rows or columns
of the result differ in size (a matrix of rank one), so do the errors: they are
matrices from the left and right times X, as large in a row and a column as the
result is there.
"""
import torch

from ops_reference import TINY, U

MUON = (3.4445, -4.7750, 2.0315)


def triples(steps, coefficients):
    return [coefficients] * steps if not hasattr(coefficients[0], "__len__") else list(coefficients)


def formula(x, steps=5, coefficients=MUON, eps=1e-7):
    """x in 64 bits."""
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (x.norm() + eps)
    for a, b, c in triples(steps, coefficients):
        A = x @ x.T
        x = a * x + (b * A + c * A @ A) @ x
    return x.T if tall else x


def _half(x, up):
    return (x * up).half().double() / up


def groups(m, n, coefs):
    """Steps of each group, as newton.cu forms them."""
    left, got = list(coefs), []
    while left:
        most = (256.0 if m >= 512 else 16.0) if not got else (16.0 if m >= 512 else 0.0)
        size, growth = 1, 1.0
        while size < len(left):
            growth *= left[size - 1][0] ** 2
            if growth > most:
                break
            size += 1
        got.append(left[:size])
        left = left[size:]
    return got


def _stored(x):
    """An m x m matrix as it is kept: fp16, times 2^6, what is above the diagonal mirrored."""
    x = _half(x, 64.0)
    return torch.triu(x) + torch.triu(x, 1).T


def rounded(x, steps=5, coefficients=MUON, eps=1e-7):
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    m, n = x.shape
    norm = x.norm() + eps
    up = 2.0 ** (8 - torch.floor(torch.log2(norm)) - 1)
    x = (x * up).half().double() / (norm * up)
    eye = torch.eye(m, dtype=x.dtype, device=x.device)
    parts = groups(m, n, triples(steps, coefficients))
    for g, part in enumerate(parts):
        A, Q = _stored(x @ x.T), None
        for i, (a, b, c) in enumerate(part):
            P = _stored(a * eye + b * A + c * A @ A)
            Q = P if Q is None else _stored(Q @ P)
            if i + 1 < len(part):
                A = _stored(_stored(A @ P) @ P)
        x = Q @ x
        if g + 1 < len(parts):
            x = _half(x, 256.0)
    return x.T if tall else x


def check(got, x, steps=5, coefficients=MUON, eps=1e-7, scale=1.0, residual=None, keep=1.0):
    x = x.double()
    want = formula(x, steps, coefficients, eps)
    rms = (rounded(x, steps, coefficients, eps) - want).norm() / want.numel() ** 0.5
    # an m x m matrix of a few elements is rounded so few times that chance decides: twice
    # what one rounding may do to each element of the result
    rms = torch.maximum(rms, 2.0 ** -11 * want.norm() / want.numel() ** 0.5)
    value = scale * want + (0 if residual is None else keep * residual.double())
    stored = U[got.dtype] * value.abs() + TINY[got.dtype] + 2.0 ** -22 * value.abs()
    d = got.double() - value
    assert torch.isfinite(d).all()
    off, most = d.norm(), 1.3 * abs(scale) * rms * want.numel() ** 0.5 + stored.norm()
    assert off <= most, f"off by {float(off / want.norm()):.3g} of the norm, at most {float(most / want.norm()):.3g}"
    size = want.norm() / want.numel() ** 0.5
    row, col = want.norm(dim=1)[:, None] / want.shape[1] ** 0.5 / size, want.norm(dim=0) / want.shape[0] ** 0.5 / size
    there = torch.clamp(torch.maximum(torch.maximum(row, col), row * col), min=1.0) if size > 0 else 1.0
    each = 10 * abs(scale) * rms * there + stored
    bad = d.abs() > each
    assert not bad.any(), f"{int(bad.sum())} elements, the worst {float((d.abs() / each).max()):.3g}"
    return float((d / scale).norm() / want.norm())
