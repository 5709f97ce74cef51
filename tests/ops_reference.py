"""64-bit reference forms of the feed-forward operators and the error bounds
their 16-bit / fp32 results are held to.

The bounds are worst-case and follow from the arithmetic, before any run:
  u        unit roundoff of the stored type: 2^-8 bf16, 2^-11 fp16, 2^-24 fp32
           (plus half the smallest subnormal of fp16, 2^-25)
  gamma(K) a K-term product summed in fp32 by 16-term tensor-core steps (or one
           by one) loses at most 2 units of 2^-24 per step, plus 16 roundings
           where partial sums are joined: (K + 32) 2^-24 covers both, times
           S = sum of |terms|
  activations: |act'| <= 1.13 for every one offered, so an error e in z moves
           act(z) by at most 1.2 e; evaluating it adds 2^-20 (1 + |z|) (fast
           exponential and division: a few units of 2^-24 times the exponent's
           argument, which is below 24 wherever the result is not negligible);
           derivatives: 2^-17 (1 + |z|) (products of up to four such factors)
  sums over rows or columns in any order: n 2^-24 sum|terms|
An intermediate that the operator documents as rounded adds u times its value.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-44}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
E = 2.0 ** -24


def gamma(k):
    return (k + 32) * E


def act(name, z):
    """(act(z), act'(z)) in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).double()
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 0.134145 * z * z)
    s = torch.sigmoid(z)
    return z * s, s * (1 + z * (1 - s))


def stored(x, dtype):
    """Rounding error bound of storing x."""
    return U[dtype] * x.abs() + TINY[dtype]


def linear(x, w, bias, activation, residual, dtype):
    """(d, bound), (z, bound); x, w (K x N), bias, residual in 64 bits."""
    z = x @ w
    S = x.abs() @ w.abs()
    e = gamma(x.shape[1]) * S
    if bias is not None:
        z = z + bias
        e = e + 2 * E * z.abs()
    d = act(activation, z)[0]
    ed = e if activation == "none" else 1.2 * e + 2.0 ** -20 * (1 + z.abs())
    if residual is not None:
        d = d + residual
        ed = ed + 2 * E * d.abs()
    return (d, ed * (1 + U[dtype]) + stored(d, dtype)), (z, e * (1 + U[dtype]) + stored(z, dtype))


def linear_backward(dd, x, w, activation, z, dtype):
    """(dx, bound), (dw, bound), (dbias, bound); dw is K x N."""
    if activation == "none":
        dz, e, er = dd, torch.zeros_like(dd), torch.zeros_like(dd)
    else:
        dz = dd * act(activation, z)[1]
        e = dd.abs() * 2.0 ** -17 * (1 + z.abs())
        er = e + stored(dz, dtype)  # the rounded dz that both products read
    a = dz.abs() + er
    dx, dw, db = dz @ w.T, x.T @ dz, dz.sum(0)
    ex = er @ w.T.abs() + gamma(w.shape[1]) * (a @ w.T.abs())
    ew = x.T.abs() @ er + gamma(x.shape[0]) * (x.T.abs() @ a)
    eb = e.sum(0) + (x.shape[0] + 8) * E * a.sum(0)
    return tuple((v, b * (1 + U[dtype]) + stored(v, dtype)) for v, b in ((dx, ex), (dw, ew), (db, eb)))


def gated(x, wg, wu, wd, activation, residual, dtype):
    """(y, bound), (g, bound), (u, bound)."""
    g, u = x @ wg, x @ wu
    eg, eu = (gamma(x.shape[1]) * (x.abs() @ w.abs()) for w in (wg, wu))
    a = act(activation, g)[0]
    ea = 1.2 * eg + 2.0 ** -20 * (1 + g.abs())
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu + 2 * E * h.abs()
    eh = eh + stored(h, dtype) + U[dtype] * eh  # h is rounded between the two kernels
    y = h @ wd
    ey = eh @ wd.abs() + gamma(wd.shape[0]) * ((h.abs() + eh) @ wd.abs())
    if residual is not None:
        y = y + residual
        ey = ey + 2 * E * y.abs()
    return tuple((v, b * (1 + U[dtype]) + stored(v, dtype)) for v, b in ((y, ey), (g, eg), (u, eu)))


def gated_backward(dy, x, wg, wu, wd, g, u, activation, dtype):
    """(dx, bound), (dwg, bound), (dwu, bound), (dwd, bound), weights in x out."""
    value, slope = act(activation, g)
    dh = dy @ wd.T
    eh = gamma(wd.shape[1]) * (dy.abs() @ wd.T.abs())
    ev, es = 2.0 ** -20 * (1 + g.abs()), 2.0 ** -17 * (1 + g.abs())
    dgv, duv, h = dh * u * slope, dh * value, value * u
    edg = u.abs() * ((dh.abs() + eh) * es + eh * slope.abs()) + 4 * E * dgv.abs()
    edu = (dh.abs() + eh) * ev + eh * value.abs() + 4 * E * duv.abs()
    ehh = ev * u.abs() + 4 * E * h.abs()
    edg, edu, ehh = (e * (1 + U[dtype]) + stored(v, dtype)  # all three are rounded workspaces
                     for e, v in ((edg, dgv), (edu, duv), (ehh, h)))
    dx = dgv @ wg.T + duv @ wu.T
    ex = edg @ wg.T.abs() + edu @ wu.T.abs() + gamma(2 * wg.shape[1]) * (
        (dgv.abs() + edg) @ wg.T.abs() + (duv.abs() + edu) @ wu.T.abs())
    out = [(dx, ex)]
    for v, e in ((dgv, edg), (duv, edu)):
        out.append((x.T @ v, x.T.abs() @ e + gamma(x.shape[0]) * (x.T.abs() @ (v.abs() + e))))
    out.append((h.T @ dy, ehh.T @ dy.abs() + gamma(x.shape[0]) * ((h.abs() + ehh).T @ dy.abs())))
    return tuple((v, b * (1 + U[dtype]) + stored(v, dtype)) for v, b in out)


def layer_norm(x, weight, bias, eps, dtype):
    """(y, bound), (mean, bound), (rstd, bound)."""
    n = x.shape[1]
    c = (n / 32 + 32) * E  # a chain per thread, then a tree
    mu = x.mean(1)
    d = x - mu[:, None]
    r = 1 / torch.sqrt((d * d).mean(1) + eps)
    emu = c * x.abs().mean(1) + E * mu.abs()
    # (x - mu) is off by emu + E |x - mu|; the variance of values all off by emu
    # gains emu^2, and its relative error is c plus that share
    er = r * (c + 8 * E + (emu * r) ** 2)
    y = d * r[:, None] * weight + bias
    ey = weight.abs() * (r[:, None] * (emu[:, None] + 2 * E * d.abs()) + d.abs() * er[:, None] * 1.01)
    ey = ey * 1.01 + 4 * E * (y.abs() + bias.abs())
    return (y, ey * (1 + U[dtype]) + stored(y, dtype)), (mu, emu), (r, er)


def layer_norm_backward(dy, x, weight, mean, rstd, dres, dtype):
    """(dx, bound), (dweight, bound), (dbias, bound); mean and rstd are inputs."""
    rows, n = x.shape
    c = (n / 32 + 32) * E
    r = rstd[:, None]
    diff = x - mean[:, None]
    xh = diff * r
    exh = 4 * E * xh.abs() + E * r * (x.abs() + mean.abs()[:, None])
    p = dy * weight
    m1, m2 = p.mean(1, keepdim=True), (p * xh).mean(1, keepdim=True)
    e1 = c * p.abs().mean(1, keepdim=True)
    e2 = c * (p * xh).abs().mean(1, keepdim=True) + (p.abs() * exh).mean(1, keepdim=True)
    dx = r * (p - m1 - xh * m2)
    ex = r * (4 * E * (p.abs() + m1.abs() + (xh * m2).abs()) + e1 + exh * m2.abs() + xh.abs() * e2)
    if dres is not None:
        dx = dx + dres
        ex = ex + 2 * E * (dx.abs() + dres.abs())
    dw, db = (dy * xh).sum(0), dy.sum(0)
    ew = (dy.abs() * exh).sum(0) + (rows + 8) * E * (dy * xh).abs().sum(0)
    eb = (rows + 8) * E * dy.abs().sum(0)
    return tuple((v, b * (1 + U[dtype]) + stored(v, dtype)) for v, b in ((dx, ex), (dw, ew), (db, eb)))


def check(got, want, what):
    """got (any type) within want = (value, bound), elementwise and finite."""
    value, bound = want
    assert tuple(got.shape) == tuple(value.shape), f"{what}: shape {tuple(got.shape)}"
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    err = (g - value).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = bad.flatten().nonzero()[0].item()
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound (worst ratio "
            f"{float((err / bound).max()):.3g}); first at {i}: got {g.flatten()[i].item()!r}, want "
            f"{value.flatten()[i].item()!r}, bound {bound.flatten()[i].item()!r}")


def make(seed, device="cuda"):
    """normal(shape, dtype, std=1, mean=0) from one seeded CPU generator."""
    gen = torch.Generator().manual_seed(seed)

    def normal(shape, dtype, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=gen) * std + mean).to(dtype).to(device)

    return normal


def pitched(x, ld, offset=0):
    """The same matrix in a wider buffer of NaN: row pitch ld, `offset` elements in."""
    rows, cols = x.shape
    buf = torch.full((offset + rows * ld + 8,), float("nan"), dtype=x.dtype, device=x.device)
    view = buf.as_strided((rows, cols), (ld, 1), offset)
    view.copy_(x)
    return view
