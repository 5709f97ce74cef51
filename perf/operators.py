"""Cases, plain forms and exact results of the feed-forward operators: layer norm, the linear layer
with its epilogue, and the gated feed-forward block, each with its backward pass.

A case names one operator in one direction; `prepare` makes what a program holds before the call,
`run` makes one pass, `exact` computes the same from the definition in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


def _ln(name, op, rows, cols, dtype, residual=False):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "residual": residual}


def _lin(name, op, M, N, K, dtype, act, bias=True, residual=False, trans_w=False, save=False):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual, "trans_w": trans_w, "save": save}


def _ffn(name, op, M, D, F, dtype, act, residual=False, trans_w=False, save=False):
    return {"name": name, "op": op, "M": M, "D": D, "F": F, "dtype": dtype, "act": act,
            "residual": residual, "trans_w": trans_w, "save": save}


def listed():
    return [
        # one new token normalised before the feed-forward block of a 4096-wide model
        _ln("ln_token", "ln_fwd", 1, 4096, "bf16"),
        # a training step's tokens, forward, with the statistics kept for the backward pass
        _ln("ln_train", "ln_fwd", 16384, 4096, "fp16"),
        # the same step's backward pass; the skip connection's gradient joins dx
        _ln("ln_train_bwd", "ln_bwd", 16384, 4096, "bf16", residual=True),
        # one new token through a projection back to the model's width, added to the residual stream
        _lin("linear_token", "linear_fwd", 1, 4096, 14336, "bf16", "none", residual=True),
        # a ragged batch through a layer whose sizes no tile divides
        _lin("linear_ragged", "linear_fwd", 1000, 1013, 997, "fp16", "gelu", residual=True),
        # a training step's tokens through the first half of a feed-forward layer; the
        # pre-activation is kept for the backward pass
        _lin("linear_train", "linear_fwd", 16384, 14336, 4096, "bf16", "gelu_tanh", save=True),
        # the gradients of a square layer with its activation
        _lin("linear_train_bwd", "linear_bwd", 8192, 4096, 4096, "bf16", "silu"),
        # one new token through the gated block: every weight is read once
        _ffn("gated_token", "gated_fwd", 1, 4096, 14336, "bf16", "silu", residual=True),
        # a serving batch of new tokens through a small model's block, weights stored out x in
        _ffn("gated_batch", "gated_fwd", 64, 1024, 4096, "fp16", "gelu_tanh", residual=True, trans_w=True),
        # a training step's forward pass; gate and up projections are kept
        _ffn("gated_train", "gated_fwd", 8192, 4096, 14336, "bf16", "silu", residual=True, save=True),
        # its backward pass: the gradients of the input and of the three weights
        _ffn("gated_train_bwd", "gated_bwd", 8192, 4096, 14336, "bf16", "silu"),
        # a short fine-tuning batch in sizes that no tile divides
        _ffn("gated_ragged_bwd", "gated_bwd", 1000, 1013, 997, "fp16", "gelu", trans_w=True),
    ]


def draw(rng):
    def size(lo, hi):  # log-uniform; half of them odd or otherwise off the tiles
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, n // 8 * 8) if rng.random() < 0.5 else n

    op = rng.choice(["ln_fwd", "ln_bwd", "linear_fwd", "linear_bwd", "gated_fwd", "gated_bwd"])
    if op.startswith("ln"):
        while True:
            rows, cols = size(1, 16384), size(64, 16384)
            if rows * cols <= 16384 * 4096:
                break
        c = _ln("", op, rows, cols, rng.choice(["bf16", "fp16", "fp32"]),
                residual=op == "ln_bwd" and rng.random() < 0.5)
    else:
        dtype, act = rng.choice(["bf16", "fp16"]), rng.choice(["relu", "gelu", "gelu_tanh", "silu"])
        if op.startswith("linear"):
            most = 2 * 16384 * 14336 * 4096 if op == "linear_fwd" else 2 * 8192 * 14336 * 4096
            while True:
                M, N, K = size(1, 16384), size(64, 14336), size(64, 14336)
                if 2 * M * N * K <= most:
                    break
            act = rng.choice(["none", act])
            c = _lin("", op, M, N, K, dtype, act, bias=rng.random() < 0.7,
                     residual=op == "linear_fwd" and rng.random() < 0.5, trans_w=rng.random() < 0.5,
                     save=op == "linear_fwd" and act != "none" and rng.random() < 0.5)
        else:
            M, D, F = size(1, 8192), size(64, 4096), size(64, 14336)
            c = _ffn("", op, M, D, F, dtype, act, residual=op == "gated_fwd" and rng.random() < 0.5,
                     trans_w=rng.random() < 0.5, save=op == "gated_fwd" and rng.random() < 0.5)
    if 3072 in c.values():  # keep off one size that is never measured
        c = {k: (3080 if v == 3072 and not isinstance(v, bool) else v) for k, v in c.items()}
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return x.mul_(std).add_(mean).to(dt)

    op, s = case["op"], {"case": dict(case)}
    if op.startswith("ln"):
        rows, cols = case["rows"], case["cols"]
        # a residual stream: a mean of its own and a few channels far larger than the rest
        x = torch.randn((rows, cols), generator=gen, device="cuda").mul_(1.5).add_(0.25)
        x[:, :: max(1, cols // 3)] *= 12.0
        s["x"] = x.to(dt)
        s["weight"], s["bias"] = normal(cols, std=0.1, mean=1.0), normal(cols, std=0.1)
        if op == "ln_bwd":
            s["dy"] = normal(rows, cols, std=0.05)
            s["dresidual"] = normal(rows, cols, std=0.05) if case["residual"] else None
            f = s["x"].float()
            s["mean"] = f.mean(1)
            s["rstd"] = (f - s["mean"][:, None]).square().mean(1).add(EPS).rsqrt()
        return s
    if op.startswith("linear"):
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = normal(M, K)
        w = normal(K, N, std=1.0 / math.sqrt(K))
        s["w"] = w.t().contiguous() if case["trans_w"] else w
        s["bias"] = normal(N, std=0.1) if case["bias"] else None
        s["residual"] = normal(M, N) if case["residual"] else None
        if op == "linear_bwd":
            s["dy"] = normal(M, N, std=0.05)
            s["z"] = None
            if case["act"] != "none":
                s["z"] = s["x"] @ w
                if case["bias"]:
                    s["z"] += s["bias"]
        return s
    M, D, F = case["M"], case["D"], case["F"]
    s["x"] = normal(M, D)
    wg, wu = normal(D, F, std=1.0 / math.sqrt(D)), normal(D, F, std=1.0 / math.sqrt(D))
    wd = normal(F, D, std=1.0 / math.sqrt(F))
    for name, w in (("wg", wg), ("wu", wu), ("wd", wd)):
        s[name] = w.t().contiguous() if case["trans_w"] else w
    s["residual"] = normal(M, D) if case["residual"] else None
    if op == "gated_bwd":
        s["dy"] = normal(M, D, std=0.05)
        s["g"], s["u"] = s["x"] @ wg, s["x"] @ wu
    return s


# -------------------------------------------------------------------- runs
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import dense_gemm_f32_gb300 as dg

    c = s["case"]
    op = c["op"]
    if op == "ln_fwd":
        return dg.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, return_stats=True)
    if op == "ln_bwd":
        return dg.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"],
                                      dresidual=s["dresidual"])
    if op == "linear_fwd":
        return dg.linear(s["x"], s["w"], bias=s["bias"], activation=c["act"], residual=s["residual"],
                         trans_w=c["trans_w"], return_preact=c["save"])
    if op == "linear_bwd":
        dx, dw, db = dg.linear_backward(s["dy"], s["x"], s["w"], activation=c["act"], preact=s["z"],
                                        trans_w=c["trans_w"], with_bias=c["bias"])
        return (dx, dw, db) if c["bias"] else (dx, dw)
    if op == "gated_fwd":
        return dg.gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], activation=c["act"],
                            residual=s["residual"], trans_w=c["trans_w"], return_saved=c["save"])
    return dg.gated_ffn_backward(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], s["g"], s["u"],
                                 activation=c["act"], trans_w=c["trans_w"])


def _act(name, z):
    if name == "relu":
        return z.clamp(min=0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    if name == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = torch.sigmoid(z)
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _run_plain(s):
    c = s["case"]
    op, dt = c["op"], _DTYPES[c["dtype"]]
    f = {k: v.float() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op == "ln_fwd":
        mean = f["x"].mean(1, keepdim=True)
        rstd = torch.rsqrt((f["x"] - mean).square().mean(1, keepdim=True) + EPS)
        y = (f["x"] - mean) * rstd * f["weight"] + f["bias"]
        return y.to(dt), mean[:, 0], rstd[:, 0]
    if op == "ln_bwd":
        xhat = (f["x"] - f["mean"][:, None]) * f["rstd"][:, None]
        gy = f["dy"] * f["weight"]
        dx = f["rstd"][:, None] * (gy - gy.mean(1, keepdim=True)
                                   - xhat * (gy * xhat).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + f["dresidual"]
        return dx.to(dt), (f["dy"] * xhat).sum(0).to(dt), f["dy"].sum(0).to(dt)
    if op.startswith("linear"):
        w = f["w"].t() if c["trans_w"] else f["w"]
        if op == "linear_fwd":
            z = f["x"] @ w
            if c["bias"]:
                z = z + f["bias"]
            d = _act(c["act"], z)
            if c["residual"]:
                d = d + f["residual"]
            return (d.to(dt), z.to(dt)) if c["save"] else d.to(dt)
        dz = f["dy"] if c["act"] == "none" else f["dy"] * _act_grad(c["act"], f["z"])
        dx, dw = dz @ w.t(), dz.t() @ f["x"] if c["trans_w"] else f["x"].t() @ dz
        return (dx.to(dt), dw.to(dt), dz.sum(0).to(dt)) if c["bias"] else (dx.to(dt), dw.to(dt))
    wg, wu, wd = (f[k].t() if c["trans_w"] else f[k] for k in ("wg", "wu", "wd"))
    if op == "gated_fwd":
        g, u = f["x"] @ wg, f["x"] @ wu
        y = (_act(c["act"], g) * u) @ wd
        if c["residual"]:
            y = y + f["residual"]
        return (y.to(dt), g.to(dt), u.to(dt)) if c["save"] else y.to(dt)
    dh, a = f["dy"] @ wd.t(), _act(c["act"], f["g"])
    du, dg_ = dh * a, dh * f["u"] * _act_grad(c["act"], f["g"])
    h = a * f["u"]
    dx = dg_ @ wg.t() + du @ wu.t()
    if c["trans_w"]:
        dws = dg_.t() @ f["x"], du.t() @ f["x"], f["dy"].t() @ h
    else:
        dws = f["x"].t() @ dg_, f["x"].t() @ du, h.t() @ f["dy"]
    return (dx.to(dt),) + tuple(w.to(dt) for w in dws)


# -------------------------------------------------------------------- work
def work(case):
    b, op = _BYTES[case["dtype"]], case["op"]
    if op.startswith("ln"):
        n, d = case["rows"] * case["cols"], case["cols"]
        if op == "ln_fwd":
            return {"bytes": b * (2 * n + 2 * d) + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": b * ((4 if case["residual"] else 3) * n + 3 * d) + 8 * case["rows"],
                "flops": 14 * n}
    if op.startswith("linear"):
        M, N, K = case["M"], case["N"], case["K"]
        n_bias = N if case["bias"] else 0
        if op == "linear_fwd":
            outs = (2 if case["save"] else 1) + (1 if case["residual"] else 0)
            return {"bytes": b * (M * K + K * N + outs * M * N + n_bias), "flops": 2 * M * N * K}
        ins = 1 if case["act"] == "none" else 2
        return {"bytes": b * (2 * M * K + 2 * K * N + ins * M * N + n_bias), "flops": 4 * M * N * K}
    M, D, F = case["M"], case["D"], case["F"]
    if op == "gated_fwd":
        return {"bytes": b * (3 * D * F + (3 if case["residual"] else 2) * M * D
                              + (2 * M * F if case["save"] else 0)),
                "flops": 6 * M * D * F}
    return {"bytes": b * (6 * D * F + 3 * M * D + 2 * M * F), "flops": 12 * M * D * F}


# ------------------------------------------------------------------- exact
def _phi(name, t):
    """(value, derivative) of an activation at t, in 64 bits."""
    if name == "none":
        return t, torch.ones_like(t)
    if name == "relu":
        on = (t > 0).double()
        return t * on, on
    if name == "silu":
        q = 1.0 / (1.0 + torch.exp(-t))
        return t * q, q + t * q * (1.0 - q)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-t / math.sqrt(2.0))
        return t * cdf, cdf + t * torch.exp(-t * t / 2.0) / math.sqrt(2.0 * math.pi)
    # 0.5 (1 + tanh v) = 1 / (1 + exp(-2 v))
    k = math.sqrt(2.0 / math.pi)
    q = 1.0 / (1.0 + torch.exp(-2.0 * k * (t + 0.044715 * t ** 3)))
    return t * q, q + t * 2.0 * q * (1.0 - q) * k * (1.0 + 0.134145 * t ** 2)


def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    v = {k: t.double() for k, t in s.items() if isinstance(t, torch.Tensor)}
    op = case["op"]
    del s
    if op.startswith("ln"):
        n = case["cols"]
        if op == "ln_fwd":
            mu = v["x"].sum(1) / n
            centred = v["x"] - mu[:, None]
            inv = 1.0 / torch.sqrt((centred * centred).sum(1) / n + EPS)
            return torch.addcmul(v["bias"], centred * inv[:, None], v["weight"]), mu, inv
        inv = v["rstd"][:, None]
        norm = (v["x"] - v["mean"][:, None]) * inv
        up = v["dy"] * v["weight"]
        dx = inv * (up - (up.sum(1)[:, None] + norm * (up * norm).sum(1)[:, None]) / n)
        if case["residual"]:
            dx += v["dresidual"]
        return dx, torch.einsum("ij,ij->j", v["dy"], norm), v["dy"].sum(0)
    if op.startswith("linear"):
        w_in_out = v["w"].T if case["trans_w"] else v["w"]
        if op == "linear_fwd":
            pre = torch.einsum("mk,kn->mn", v["x"], w_in_out)
            if case["bias"]:
                pre += v["bias"]
            out = _phi(case["act"], pre)[0]
            if case["residual"]:
                out = out + v["residual"]
            return (out, pre) if case["save"] else out
        up = v["dy"] if case["act"] == "none" else v["dy"] * _phi(case["act"], v["z"])[1]
        dw = torch.einsum("mk,mn->kn", v["x"], up)
        got = torch.einsum("mn,kn->mk", up, w_in_out), dw.T if case["trans_w"] else dw
        return got + (up.sum(0),) if case["bias"] else got
    w = {k: v[k].T if case["trans_w"] else v[k] for k in ("wg", "wu", "wd")}
    if op == "gated_fwd":
        gate, lin = torch.einsum("md,df->mf", v["x"], w["wg"]), torch.einsum("md,df->mf", v["x"], w["wu"])
        out = torch.einsum("mf,fd->md", _phi(case["act"], gate)[0] * lin, w["wd"])
        if case["residual"]:
            out += v["residual"]
        return (out, gate, lin) if case["save"] else out
    value, slope = _phi(case["act"], v["g"])
    dh = torch.einsum("md,fd->mf", v["dy"], w["wd"])
    dgate, dlin = dh * v["u"] * slope, dh * value
    dx = torch.einsum("mf,df->md", dgate, w["wg"]) + torch.einsum("mf,df->md", dlin, w["wu"])
    dws = (torch.einsum("md,mf->df", v["x"], dgate), torch.einsum("md,mf->df", v["x"], dlin),
           torch.einsum("mf,md->fd", value * v["u"], v["dy"]))
    return (dx,) + tuple(t.T if case["trans_w"] else t for t in dws)
