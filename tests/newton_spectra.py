"""Matrices on which rounding shows in an orthogonalised update, and the limit that the
operator documents for them: steep spectra, a few directions over a floor, matrices of low
rank, and such with few distinct values, whose elements round alike.

The limit, for five steps of the usual coefficients: an update is off by at most LIMIT of its
norm.  Most of it is the rounding of the iterate to fp16 after the first two steps, half a step
of 2^-10 at most, 2^-11 / sqrt 3 of an element in the root mean square.  Where X has no direction of its
own the three steps left enlarge that by a^3 = 40.87; a matrix of rank one has a norm of 1.114 then
and of 0.697 at the end, so 40.87 x 2.82e-4 x 1.114 / 0.697 = 0.0184, with elements just above
a power of two (0.0121 with mantissas spread evenly).  The iterate's rounding one and two steps later is enlarged by
a^2 and a, 0.0054 and 0.0015 added in squares: 0.0193.  The m x m matrices, exact where X has no
direction, turn directions by a few roundings of 2^-12: 0.02 in all.

FEW, for a smaller side of 2 to 7: a handful of elements may all round the same way.  In the first group A is
off by 2^-11 of its largest singular value then, its successor by a^2 = 11.9 times that where a singular
value is small, and by as much again from the product in between, 0.009; P by b = 4.8 times this, 1.2% of
a; and each of the three steps after it enlarges a relative error by up to 1.6, the steepest slope of
the polynomial between 0.68 and 1.13: 0.05, beside the 0.0193 above.
"""
import torch

LIMIT = 0.02
FEW = 0.07


def _spread(m, n, sizes, gen):
    """Singular values `sizes` in directions drawn at random."""
    u = torch.linalg.qr(torch.randn((m, len(sizes)), dtype=torch.float64, generator=gen))[0]
    v = torch.linalg.qr(torch.randn((n, len(sizes)), dtype=torch.float64, generator=gen))[0]
    return (u * sizes) @ v.T


def _two_valued(m, n, ratio, second, gen):
    """Rank two, the left vectors constant on each half of the rows."""
    u, w = torch.ones(m, dtype=torch.float64), torch.full((m,), ratio, dtype=torch.float64)
    u[m // 2:], w[m // 2:] = ratio, -1.0
    v = torch.linalg.qr(torch.randn((n, 2), dtype=torch.float64, generator=gen))[0]
    return torch.outer(u / u.norm(), v[:, 0]) + second * torch.outer(w / w.norm(), v[:, 1])


NAMES = ("flat", "i^-1", "i^-1.5", "i^-2", "i^-3", "i^-4", "eight over a floor", "one over a floor", "rank one",
         "rank three", "equal rows", "two values, 1.7", "two values, 1.3")


def make(name, rows, cols, dtype, seed=0):
    """The matrix, on the CPU, its largest element 1 (taller than wide: the transposed one)."""
    m, n = min(rows, cols), max(rows, cols)
    gen = torch.Generator().manual_seed(seed)
    i = torch.arange(1, m + 1, dtype=torch.float64)
    if name.startswith("i^"):
        x = _spread(m, n, i ** float(name[2:]), gen)
    elif name == "flat":
        x = _spread(m, n, torch.ones_like(i), gen)
    elif name == "eight over a floor":
        x = _spread(m, n, torch.where(i <= 8, 1.0, 1e-3), gen)
    elif name == "one over a floor":
        x = _spread(m, n, torch.where(i <= 1, 1.0, 1e-2), gen)
    elif name == "rank one":
        x = _spread(m, n, i[:1], gen)
    elif name == "rank three":
        x = _spread(m, n, torch.tensor([1.0, 0.3, 0.01], dtype=torch.float64)[:m], gen)
    elif name == "equal rows":
        x = torch.randn((1, n), dtype=torch.float64, generator=gen).expand(m, n)
    else:
        ratio = float(name.split()[-1])
        x = _two_valued(m, n, ratio, 0.01 if ratio > 1.5 else 0.1, gen)
    x = (x / x.abs().max()).to(dtype)
    return x.T.contiguous() if rows > cols else x.contiguous()
