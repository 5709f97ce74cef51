"""64-bit reference forms of the products in 8-bit integers, and the bounds
their results are held to (derived before any run; ops_reference.py has the
common part).

Integers of 16-bit rows are compared exactly: round(127 x / top) in 64 bits is
exact, for 127 x is and a quotient of an 18-bit and an 11-bit integer that is
not a half of an odd number is at least 2^-20 of itself from one.  A sum of
integer products is exact while sum |q w| <= 2^24; beyond, each of its K / 16
steps and of the joins of its parts loses at most 2 units of 2^-24 of that.
Scaling rounds twice, and the row's scale was rounded once.  Hidden units are
float32, off by e from the reference's; where 127 h / top lies that close to a
half, the integer may be the neighbour: one scale more.
"""
import torch

import ops_reference as ref
from ops_reference import E, U


def quantize(x):
    """(q, scale) of rows in 64 bits; zeros, and the scale itself, where it is not finite or 0."""
    x = x.double()
    top = x.abs().amax(1) if x.shape[1] else torch.zeros_like(x[:, :0].sum(1))
    ok = torch.isfinite(top) & (top > 0)
    q = torch.round(127.0 * x / torch.where(ok, top, torch.ones_like(top))[:, None])
    return torch.where(ok[:, None], q, torch.zeros_like(q)), top / 127.0


def product(q, scale, w, w_scale):
    """(z, bound): integers q (M x K) and w (N x K) in 64 bits with their scales."""
    acc, S = q @ w.T, q.abs() @ w.abs().T
    e = torch.where(S <= 2.0 ** 24, torch.zeros_like(S), 2 * E * (q.shape[1] / 16 + 16) * S)
    s = scale[:, None] * w_scale
    z = acc * s
    return z, e * s + 4 * E * z.abs()


def finish(z, e, bias, activation, residual, dtype):
    if bias is not None:
        z = z + bias
        e = e + 2 * E * z.abs()
    d = ref.act(activation, z)[0]
    ed = e if activation == "none" else 1.2 * e + 2.0 ** -20 * (1 + z.abs())
    if residual is not None:
        d = d + residual
        ed = ed + 2 * E * d.abs()
    return d, ed * (1 + U[dtype]) + ref.stored(d, dtype)


def linear(q, scale, w, w_scale, bias, activation, residual, dtype):
    return finish(*product(q, scale, w, w_scale), bias, activation, residual, dtype)


def gated(x, wg, sg, wu, su, wd, sd, activation, residual, dtype):
    q, s = quantize(x)
    g, eg = product(q, s, wg, sg)
    u, eu = product(q, s, wu, su)
    a = ref.act(activation, g)[0]
    ea = 1.2 * eg + 2.0 ** -20 * (1 + g.abs())
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu + 2 * E * h.abs()
    q2, s2 = quantize(h)
    top = 127.0 * s2
    etop = eh.amax(1) if h.shape[1] else torch.zeros_like(top)
    # how far 127 h / top may be off, and whether a border is as near
    t = 127.0 * h / torch.where(top > 0, top, torch.ones_like(top))[:, None]
    et = 127.0 * eh / torch.where(top > 0, top, torch.ones_like(top))[:, None]
    et = et + t.abs() * (etop / torch.where(top > 0, top, torch.ones_like(top)))[:, None] + 4 * E * t.abs()
    near = (((t - torch.floor(t)) - 0.5).abs() <= et).double() + torch.floor(et)
    eq = near * s2[:, None] + q2.abs() * (etop / 127.0 + E * s2)[:, None]
    z, e = product(q2, s2, wd, sd)
    e = e * 1.01 + eq @ (wd.abs() * sd[:, None]).T
    return finish(z, e, None, "none", residual, dtype)
