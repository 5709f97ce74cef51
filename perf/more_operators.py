"""Cases, plain forms and exact results of the 8-bit integer products (the linear layer and the gated
feed-forward block with weights held in 8 bits and a scale for each token and channel) and of the
orthogonalisation of a weight update by Newton-Schulz products.

A case names one operator; `prepare` makes what a program holds before the call, `run` makes one
pass, `exact` computes the same from the definition in 64 bits.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)  # of the Muon optimiser's iteration
EPS = 1e-7


def _lin(name, M, N, K, dtype, act="none", bias=False, residual=False, given=False):
    # given: the tokens are in 8 bits already, quantised once for several products
    return {"name": name, "op": "linear_int8", "M": M, "N": N, "K": K, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual, "given": given}


def _ffn(name, M, D, F, dtype, act, residual=False):
    return {"name": name, "op": "gated_int8", "M": M, "D": D, "F": F, "dtype": dtype, "act": act,
            "residual": residual}


def _orth(name, rows, cols, dtype, update=False, steps=5):
    # update: the result joins the weights, w <- (1 - lr decay) w - lr scale orthogonalised
    return {"name": name, "op": "orthogonalize", "rows": rows, "cols": cols, "dtype": dtype,
            "update": update, "steps": steps}


def listed():
    return [
        # one new token through a projection up from a 4096-wide model
        _lin("int8_token", 1, 14336, 4096, "bf16"),
        # a serving batch of new tokens back down to the model's width, onto the residual stream
        _lin("int8_batch", 64, 4096, 14336, "bf16", residual=True),
        # a ragged batch through a layer whose sizes no tile divides, tokens given in 8 bits
        _lin("int8_ragged", 1000, 1013, 997, "fp16", "gelu", bias=True, residual=True, given=True),
        # a long prompt through a layer with its activation
        _lin("int8_prompt", 8192, 14336, 4096, "bf16", "gelu_tanh", bias=True),
        # one new token through the gated block: every weight is read once
        _ffn("gated_int8_token", 1, 4096, 14336, "bf16", "silu", residual=True),
        # a serving batch of new tokens through a small model's block
        _ffn("gated_int8_batch", 64, 1024, 4096, "fp16", "gelu_tanh", residual=True),
        # a short prompt
        _ffn("gated_int8_short", 512, 4096, 14336, "bf16", "silu", residual=True),
        # a long one
        _ffn("gated_int8_prompt", 8192, 4096, 14336, "bf16", "silu", residual=True),
        # the update of a small block's gate projection
        _orth("orthogonal_small", 512, 1408, "bf16"),
        # a matrix that no tile divides, more rows than columns, in half precision
        _orth("orthogonal_ragged", 1013, 997, "fp16", update=True),
        # a square layer's update, applied to its weights
        _orth("orthogonal_square", 4096, 4096, "bf16", update=True),
        # the update of a large block's down projection, applied to its weights
        _orth("orthogonal_large", 14336, 4096, "bf16", update=True),
    ]


def draw(rng):
    def size(lo, hi):  # log-uniform; half of them odd or otherwise off the tiles
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, n // 16 * 16) if rng.random() < 0.5 else n

    op = rng.choice(["linear_int8", "gated_int8", "orthogonalize"])
    dtype = rng.choice(["bf16", "fp16"])
    act = rng.choice(["relu", "gelu", "gelu_tanh", "silu"])
    if op == "linear_int8":
        c = _lin("", size(1, 8192), size(64, 14336), size(64, 14336), dtype, rng.choice(["none", act]),
                 bias=rng.random() < 0.5, residual=rng.random() < 0.5, given=rng.random() < 0.4)
    elif op == "gated_int8":
        c = _ffn("", size(1, 8192), size(64, 4096), size(64, 14336), dtype, act, residual=rng.random() < 0.5)
    else:
        rows, cols = size(64, 14336), size(64, 4096)
        if rng.random() < 0.5:
            rows, cols = cols, rows
        c = _orth("", rows, cols, dtype, update=rng.random() < 0.5, steps=rng.choice([3, 5, 5, 6]))
        if c["steps"] == 6 and rows * cols > 4096 * 8192:
            c["steps"] = 5  # no dearer than the largest listed case
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _quantised(w):
    """8-bit integers of a matrix with a scale for each row, as a program holds its weights."""
    w = w.float()
    scale = w.abs().amax(1).clamp(min=1e-30) / 127.0
    return torch.round(w / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)

    op, s = case["op"], {"case": dict(case)}
    if op == "orthogonalize":
        rows, cols = case["rows"], case["cols"]
        # a gradient: a few strong directions over a floor of noise
        rank = max(1, min(rows, cols) // 8)
        g = normal(rows, rank) @ normal(rank, cols, std=1.0 / math.sqrt(rank))
        s["g"] = g.add_(normal(rows, cols, std=0.3)).mul_(1e-3).to(dt)
        if case["update"]:
            s["w"] = normal(rows, cols, std=1.0 / math.sqrt(rows)).to(dt)
        return s
    K = case["K"] if op == "linear_int8" else case["D"]
    # activations: a few channels far larger than the rest
    x = normal(case["M"], K)
    x[:, :: max(1, K // 3)] *= 8.0
    s["x"] = x.to(dt)
    if op == "linear_int8":
        M, N = case["M"], case["N"]
        s["w"], s["w_scale"] = _quantised(normal(N, K, std=1.0 / math.sqrt(K)))
        s["bias"] = normal(N, std=0.1).to(dt) if case["bias"] else None
        s["residual"] = normal(M, N).to(dt) if case["residual"] else None
        s["x_scale"] = None
        if case["given"]:
            s["x"], s["x_scale"] = _quantised(s["x"])
        return s
    F = case["F"]
    s["wg"], s["sg"] = _quantised(normal(F, K, std=1.0 / math.sqrt(K)))
    s["wu"], s["su"] = _quantised(normal(F, K, std=1.0 / math.sqrt(K)))
    s["wd"], s["sd"] = _quantised(normal(K, F, std=1.0 / math.sqrt(F)))
    s["residual"] = normal(case["M"], K).to(dt) if case["residual"] else None
    return s


def _lr(case):
    """(scale of the orthogonalised update, scale of the weights) of one step."""
    lr, decay = 0.02, 0.1
    return -lr * math.sqrt(max(1.0, case["rows"] / case["cols"])), 1.0 - lr * decay


# -------------------------------------------------------------------- runs
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import dense_gemm_f32_gb300 as dg

    c = s["case"]
    if c["op"] == "linear_int8":
        return dg.linear_int8(s["x"], s["w"], s["w_scale"], bias=s["bias"], activation=c["act"],
                              residual=s["residual"], x_scale=s["x_scale"], dtype=_DTYPES[c["dtype"]])
    if c["op"] == "gated_int8":
        return dg.gated_ffn_int8(s["x"], s["wg"], s["sg"], s["wu"], s["su"], s["wd"], s["sd"],
                                 activation=c["act"], residual=s["residual"])
    if c["update"]:
        scale, keep = _lr(c)
        return dg.orthogonalize(s["g"], steps=c["steps"], coefficients=COEFFICIENTS, eps=EPS, scale=scale,
                                residual=s["w"], residual_scale=keep)
    return dg.orthogonalize(s["g"], steps=c["steps"], coefficients=COEFFICIENTS, eps=EPS)


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


def _tokens(x):
    """Each row as integers of at most 127 in size, round(127 x / largest), and its scale; the
    quotient in 64 bits, because a half lies next to the border of two integers."""
    largest = x.float().abs().amax(1, keepdim=True)
    q = torch.round(x.double() * 127.0 / largest.double().clamp(min=1e-300))
    return q.float(), largest / 127.0


def _run_plain(s):
    c = s["case"]
    dt = _DTYPES[c["dtype"]]
    if c["op"] == "orthogonalize":
        g = s["g"].float()
        x = g.t() if c["rows"] > c["cols"] else g
        x = x / (torch.sqrt(x.square().sum()) + EPS)
        a, b, k = COEFFICIENTS
        for _ in range(c["steps"]):
            gram = x @ x.t()
            x = a * x + (b * gram + k * (gram @ gram)) @ x
        x = x.t() if c["rows"] > c["cols"] else x
        if c["update"]:
            scale, keep = _lr(c)
            x = keep * s["w"].float() + scale * x
        return x.to(dt).contiguous()
    if c["op"] == "linear_int8":
        q, scale = (s["x"].float(), s["x_scale"][:, None]) if c["given"] else _tokens(s["x"])
        z = (q @ s["w"].float().t()) * scale * s["w_scale"]
        if c["bias"]:
            z = z + s["bias"].float()
        y = _act(c["act"], z)
        if c["residual"]:
            y = y + s["residual"].float()
        return y.to(dt)
    q, scale = _tokens(s["x"])
    gate = (q @ s["wg"].float().t()) * scale * s["sg"]
    up = (q @ s["wu"].float().t()) * scale * s["su"]
    q, scale = _tokens(_act(c["act"], gate) * up)
    y = (q @ s["wd"].float().t()) * scale * s["sd"]
    if c["residual"]:
        y = y + s["residual"].float()
    return y.to(dt)


# -------------------------------------------------------------------- work
def work(case):
    b = _BYTES[case["dtype"]]
    if case["op"] == "orthogonalize":
        m, n = sorted((case["rows"], case["cols"]))
        t = case["steps"]
        # With the smaller side m: X X^T is symmetric (m m n operations for half of it), as are its
        # polynomials (m^3 each).  Either every step forms X X^T, its square and the product with X,
        # or the steps stay among m x m matrices (the polynomial, the product of all polynomials so
        # far, and two products for the next step's X X^T) between one X X^T and one product with X.
        each = t * (3 * m * m * n + m ** 3)
        inner = 3 * m * m * n + (max(0, 4 * t - 3)) * m ** 3
        return {"bytes": b * (3 if case["update"] else 2) * m * n, "flops": min(each, inner)}
    M = case["M"]
    if case["op"] == "linear_int8":
        N, K = case["N"], case["K"]
        return {"bytes": N * K + 4 * N + (M * K + 4 * M if case["given"] else b * M * K)
                + b * ((2 if case["residual"] else 1) * M * N + (N if case["bias"] else 0)),
                "flops": 2 * M * N * K}
    D, F = case["D"], case["F"]
    return {"bytes": 3 * D * F + 4 * (2 * F + D) + b * (3 if case["residual"] else 2) * M * D,
            "flops": 6 * M * D * F}


# ------------------------------------------------------------------- exact
def _phi(name, t):
    """An activation in 64 bits."""
    if name == "none":
        return t
    if name == "relu":
        return t * (t > 0).double()
    if name == "silu":
        return t / (1.0 + torch.exp(-t))
    if name == "gelu":
        return t * 0.5 * torch.special.erfc(-t / math.sqrt(2.0))
    k = math.sqrt(2.0 / math.pi)  # 0.5 (1 + tanh v) = 1 / (1 + exp(-2 v))
    return t / (1.0 + torch.exp(-2.0 * k * (t + 0.044715 * t ** 3)))


def _rows_in_8_bits(t):
    """The values that rows in 8 bits stand for: multiples of max|t| / 127, the nearest ones."""
    top = torch.amax(torch.abs(t), dim=1)
    unit = torch.where(top > 0, top, torch.ones_like(top))[:, None]
    return torch.round(127.0 * t / unit) * (top[:, None] / 127.0)


def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    v = {k: t.double() for k, t in s.items() if isinstance(t, torch.Tensor)}
    del s
    if case["op"] == "orthogonalize":
        x = v.pop("g")
        wide = case["cols"] >= case["rows"]
        x /= x.norm() + EPS
        a, b, k = COEFFICIENTS
        for _ in range(case["steps"]):
            if wide:
                p = torch.einsum("ik,jk->ij", x, x)
                p = torch.addmm(p, p, p, beta=b, alpha=k)
                x = torch.addmm(x, p, x, beta=a)
            else:
                p = torch.einsum("ki,kj->ij", x, x)
                p = torch.addmm(p, p, p, beta=b, alpha=k)
                x = torch.addmm(x, x, p, beta=a)
        if case["update"]:
            scale, keep = _lr(case)
            x = torch.add(keep * v["w"], x, alpha=scale)
        return x
    if case["op"] == "linear_int8":
        x = v["x"] * v["x_scale"][:, None] if case["given"] else _rows_in_8_bits(v["x"])
        z = torch.einsum("mk,nk->mn", x, v["w"] * v["w_scale"][:, None])
        if case["bias"]:
            z += v["bias"]
        z = _phi(case["act"], z)
        return z + v["residual"] if case["residual"] else z
    x = _rows_in_8_bits(v["x"])
    gate = torch.einsum("md,fd->mf", x, v["wg"] * v["sg"][:, None])
    up = torch.einsum("md,fd->mf", x, v["wu"] * v["su"][:, None])
    hidden = _rows_in_8_bits(_phi(case["act"], gate) * up)
    out = torch.einsum("mf,df->md", hidden, v["wd"] * v["sd"][:, None])
    return out + v["residual"] if case["residual"] else out
