"""The feed-forward operators over torch CUDA tensors: layer norm, the linear
layer with bias, activation and residual in its epilogue, and the gated
feed-forward block, each with its backward pass.

Like `matmul`, these only check shapes and types, derive pointers, leading
dimensions and the stream, allocate outputs and workspaces, and raise on a
non-zero status; all arithmetic runs in the library's kernels.  Activations
may have any number of leading dimensions that flatten into rows without a
copy; the last dimension is contiguous.  Outputs are allocated on the stream
the call runs on (`stream`, default the current one); tensors made on another
stream must be ready there, as for any torch call.
"""
import torch

from . import _lib
from ._lib import (
    ACT_GELU, ACT_GELU_TANH, ACT_NONE, ACT_RELU, ACT_SILU, DTYPE_BF16, DTYPE_F16, DTYPE_F32, OK,
    OP_N, OP_T,
)

ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH,
               "silu": ACT_SILU}

_HALF = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
_FLOAT = {**_HALF, torch.float32: DTYPE_F32}


def _check(status, what):
    if status != OK:
        from . import DgemmError

        raise DgemmError(status, what)


def _on(stream, x):
    """(raw handle, context in which outputs are allocated) for `stream`."""
    if stream is None:
        return torch.cuda.current_stream(x.device).cuda_stream, None
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream, device=x.device)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _in(context, f):
    if context is None:
        return f()
    with context:
        return f()


def _dtype(table, name, x):
    code = table.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} takes {', '.join(str(d) for d in table)}, got {x.dtype}")
    return code


def _rows(x, name, dtype, cols=None):
    """(rows, cols, leading dimension) of x with its leading dimensions flattened."""
    if x.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {x.dtype}")
    if x.dim() == 0:
        raise ValueError(f"{name}: expected at least one dimension")
    c = x.shape[-1]
    if cols is not None and c != cols:
        raise ValueError(f"{name}: the last dimension is {c}, expected {cols}")
    if x.dim() == 2:
        r = x.shape[0]
    else:
        r = x.numel() // c if c else x.shape[:-1].numel()
        try:
            x = x.view(r, c)
        except RuntimeError:
            raise ValueError(f"{name}: the leading dimensions do not flatten into rows") from None
    if c > 1 and r > 0 and x.stride(1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return r, c, x.stride(0) if r > 1 else max(c, 1)


def _like(x, name, dtype, rows, cols):
    """Leading dimension of x, which has to be rows x cols."""
    r, c, ld = _rows(x, name, dtype, cols)
    if r != rows:
        raise ValueError(f"{name}: {r} rows, expected {rows}")
    return ld


def _optional(x, name, dtype, rows, cols):
    """(pointer, leading dimension) of an optional matrix."""
    if x is None:
        return 0, max(cols, 1)
    return x.data_ptr(), _like(x, name, dtype, rows, cols)


def _vector(x, name, dtype, n):
    if x is None:
        return 0
    if x.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {x.dtype}")
    if x.dim() != 1 or x.shape[0] != n:
        raise ValueError(f"{name}: expected {n} elements, got {tuple(x.shape)}")
    if n > 1 and x.stride(0) != 1:
        raise ValueError(f"{name}: must be contiguous")
    return x.data_ptr()


def _weight(w, name, dtype, inner, outer, trans_w):
    """Leading dimension of a weight: inner x outer, or outer x inner when trans_w."""
    want = (outer, inner) if trans_w else (inner, outer)
    if w.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {w.dtype}")
    if tuple(w.shape) != want:
        raise ValueError(f"{name}: expected {want[0]}x{want[1]}, got {tuple(w.shape)}")
    return _like(w, name, dtype, *want)


def _activation(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)}, got {name!r}")
    return code


def _pitched(rows, cols, like):
    """A rows x cols workspace whose rows start on 16-byte boundaries."""
    ld = (cols + 7) // 8 * 8
    return torch.empty((rows, ld), dtype=like.dtype, device=like.device), max(ld, 1)


def layer_norm(x, weight=None, bias=None, eps=1e-5, return_stats=False, out=None, stream=None):
    """y = (x - mean) rstd weight + bias over the last dimension.

    x: (..., n) bfloat16, float16 or float32.  weight, bias: n elements of the
    same type, or None.  out: optional tensor of x's shape and type to write.
    Returns y, or (y, mean, rstd) with the float32 statistics of every row
    (shape x.shape[:-1]) that layer_norm_backward takes.
    """
    dt = _dtype(_FLOAT, "layer_norm", x)
    rows, cols, ldx = _rows(x, "x", x.dtype)
    pw, pb = _vector(weight, "weight", x.dtype, cols), _vector(bias, "bias", x.dtype, cols)
    if out is not None and out.shape != x.shape:
        raise ValueError(f"out: expected {tuple(x.shape)}, got {tuple(out.shape)}")
    handle, context = _on(stream, x)

    def allocate():
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device) if out is None else out
        s = torch.empty((2,) + x.shape[:-1], dtype=torch.float32, device=x.device) if return_stats else None
        return y, s

    y, stats = _in(context, allocate)
    mean, rstd = (stats[0], stats[1]) if return_stats else (None, None)
    st = _lib.dgemm_layer_norm(dt, rows, cols, eps, x.data_ptr(), ldx, pw, pb, y.data_ptr(),
                               _like(y, "out", x.dtype, rows, cols),
                               mean.data_ptr() if return_stats else 0,
                               rstd.data_ptr() if return_stats else 0, handle)
    _check(st, "layer_norm")
    return (y, mean, rstd) if return_stats else y


def layer_norm_backward(dy, x, weight, mean, rstd, dresidual=None, stream=None):
    """(dx, dweight, dbias) of layer_norm.

    mean, rstd: what layer_norm returned.  dresidual: a gradient of x's shape
    that joins dx (that of a skip connection around the norm), or None.  weight
    may be None (then 1; dweight is still returned).
    """
    dt = _dtype(_FLOAT, "layer_norm_backward", x)
    rows, cols, ldx = _rows(x, "x", x.dtype)
    lddy = _like(dy, "dy", x.dtype, rows, cols)
    pr, lddr = _optional(dresidual, "dresidual", x.dtype, rows, cols)
    pw = _vector(weight, "weight", x.dtype, cols)
    pm = _vector(mean.reshape(-1), "mean", torch.float32, rows)
    ps = _vector(rstd.reshape(-1), "rstd", torch.float32, rows)
    handle, context = _on(stream, x)

    def allocate():
        return (torch.empty(x.shape, dtype=x.dtype, device=x.device),
                torch.empty((2, cols), dtype=x.dtype, device=x.device))

    dx, grads = _in(context, allocate)
    dw, db = grads[0], grads[1]
    st = _lib.dgemm_layer_norm_backward(dt, rows, cols, dy.data_ptr(), lddy, x.data_ptr(), ldx, pw,
                                        pm, ps, pr, lddr, dx.data_ptr(), max(cols, 1),
                                        dw.data_ptr(), db.data_ptr(), handle)
    _check(st, "layer_norm_backward")
    return dx, dw, db


def linear(x, w, bias=None, activation="none", residual=None, trans_w=False, return_preact=False,
           out=None, stream=None):
    """act(x @ op(w) + bias) + residual in one kernel.

    x: (..., K) bfloat16 or float16; w: K x N, or N x K with trans_w; bias: N
    elements; residual: (..., N); all of x's type.  out: optional (..., N)
    tensor to write, which may be `residual` itself.  Returns d, or
    (d, preact) with preact = x @ op(w) + bias, which linear_backward takes.
    """
    dt, act = _dtype(_HALF, "linear", x), _activation(activation)
    if w.dim() != 2:
        raise ValueError("w: expected a 2-D matrix")
    M, K, ldx = _rows(x, "x", x.dtype)
    N = w.shape[0] if trans_w else w.shape[1]
    ldw = _weight(w, "w", x.dtype, K, N, trans_w)
    pb = _vector(bias, "bias", x.dtype, N)
    pr, ldr = _optional(residual, "residual", x.dtype, M, N)
    shape = x.shape[:-1] + (N,)
    if out is not None and out.shape != shape:
        raise ValueError(f"out: expected {tuple(shape)}, got {tuple(out.shape)}")
    handle, context = _on(stream, x)

    def allocate():
        d = torch.empty(shape, dtype=x.dtype, device=x.device) if out is None else out
        return d, torch.empty(shape, dtype=x.dtype, device=x.device) if return_preact else None

    d, z = _in(context, allocate)
    st = _lib.dgemm_linear(dt, act, OP_T if trans_w else OP_N, M, N, K, x.data_ptr(), ldx,
                           w.data_ptr(), ldw, pb, pr, ldr, d.data_ptr(),
                           _like(d, "out", x.dtype, M, N), z.data_ptr() if return_preact else 0,
                           max(N, 1), handle)
    _check(st, "linear")
    return (d, z) if return_preact else d


def linear_backward(dd, x, w, activation="none", preact=None, trans_w=False, with_bias=True,
                    stream=None):
    """(dx, dw, dbias) of linear; dbias is None without with_bias.

    dd: the gradient of linear's result (also that of its residual).  preact:
    what linear(..., return_preact=True) returned; needed unless activation is
    "none".
    """
    dt, act = _dtype(_HALF, "linear_backward", x), _activation(activation)
    if w.dim() != 2:
        raise ValueError("w: expected a 2-D matrix")
    M, K, ldx = _rows(x, "x", x.dtype)
    N = w.shape[0] if trans_w else w.shape[1]
    ldw = _weight(w, "w", x.dtype, K, N, trans_w)
    lddd = _like(dd, "dd", x.dtype, M, N)
    if act != ACT_NONE and preact is None:
        raise ValueError(f"preact is needed for activation {activation!r}")
    pz, ldz = _optional(preact if act != ACT_NONE else None, "preact", x.dtype, M, N)
    handle, context = _on(stream, x)

    def allocate():
        dz, lddz = _pitched(M, N, x) if act != ACT_NONE else (None, max(N, 1))
        return (torch.empty(x.shape, dtype=x.dtype, device=x.device),
                torch.empty(w.shape, dtype=x.dtype, device=x.device),
                torch.empty((N,), dtype=x.dtype, device=x.device) if with_bias else None, dz, lddz)

    dx, dw, db, dz, lddz = _in(context, allocate)
    st = _lib.dgemm_linear_backward(dt, act, OP_T if trans_w else OP_N, M, N, K, dd.data_ptr(),
                                    lddd, x.data_ptr(), ldx, w.data_ptr(), ldw, pz, ldz,
                                    dz.data_ptr() if dz is not None else 0, lddz, dx.data_ptr(),
                                    max(K, 1), dw.data_ptr(), max(w.shape[1], 1),
                                    db.data_ptr() if with_bias else 0, handle)
    _check(st, "linear_backward")
    return dx, dw, db


def _block(what, x, w_gate, w_up, w_down, trans_w):
    """Sizes and leading dimensions of a gated block's input and weights."""
    dt = _dtype(_HALF, what, x)
    for name, w in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        if w.dim() != 2:
            raise ValueError(f"{name}: expected a 2-D matrix")
    M, D, ldx = _rows(x, "x", x.dtype)
    F = w_gate.shape[0] if trans_w else w_gate.shape[1]
    ldwg = _weight(w_gate, "w_gate", x.dtype, D, F, trans_w)
    ldwu = _weight(w_up, "w_up", x.dtype, D, F, trans_w)
    ldwd = _weight(w_down, "w_down", x.dtype, F, D, trans_w)
    return dt, M, D, F, ldx, ldwg, ldwu, ldwd


def gated_ffn(x, w_gate, w_up, w_down, activation="silu", residual=None, trans_w=False,
              return_saved=False, out=None, stream=None):
    """(act(x @ op(w_gate)) * (x @ op(w_up))) @ op(w_down) + residual.

    x: (..., D) bfloat16 or float16.  w_gate, w_up: D x F and w_down: F x D, or
    their transposes with trans_w.  residual: of x's shape; out may be it.
    Returns y, or (y, g, u) with the two projections, (..., F), which
    gated_ffn_backward takes.
    """
    act = _activation(activation)
    dt, M, D, F, ldx, ldwg, ldwu, ldwd = _block("gated_ffn", x, w_gate, w_up, w_down, trans_w)
    pr, ldr = _optional(residual, "residual", x.dtype, M, D)
    if out is not None and out.shape != x.shape:
        raise ValueError(f"out: expected {tuple(x.shape)}, got {tuple(out.shape)}")
    handle, context = _on(stream, x)

    def allocate():
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device) if out is None else out
        saved = [torch.empty(x.shape[:-1] + (F,), dtype=x.dtype, device=x.device)
                 for _ in range(2 if return_saved else 0)]
        return y, saved, _pitched(M, F, x)

    y, saved, (h, ldh) = _in(context, allocate)
    pg, pu = (saved[0].data_ptr(), saved[1].data_ptr()) if return_saved else (0, 0)
    st = _lib.dgemm_gated_ffn(dt, act, OP_T if trans_w else OP_N, M, D, F, x.data_ptr(), ldx,
                              w_gate.data_ptr(), ldwg, w_up.data_ptr(), ldwu, w_down.data_ptr(),
                              ldwd, pr, ldr, h.data_ptr(), ldh, pg, max(F, 1), pu, max(F, 1),
                              y.data_ptr(), _like(y, "out", x.dtype, M, D), handle)
    _check(st, "gated_ffn")
    return (y, saved[0], saved[1]) if return_saved else y


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, g, u, activation="silu", trans_w=False,
                       stream=None):
    """(dx, dw_gate, dw_up, dw_down) of gated_ffn from its saved g and u.

    dy: the gradient of gated_ffn's result (also that of its residual).
    """
    act = _activation(activation)
    dt, M, D, F, ldx, ldwg, ldwu, ldwd = _block("gated_ffn_backward", x, w_gate, w_up, w_down,
                                                trans_w)
    lddy = _like(dy, "dy", x.dtype, M, D)
    ldg, ldu = _like(g, "g", x.dtype, M, F), _like(u, "u", x.dtype, M, F)
    handle, context = _on(stream, x)

    def allocate():
        return ([torch.empty(t.shape, dtype=x.dtype, device=x.device) for t in (x, w_gate, w_up, w_down)],
                [_pitched(M, F, x) for _ in range(3)])

    (dx, dwg, dwu, dwd), ((h, ldh), (dg, lddg), (du, lddu)) = _in(context, allocate)
    up, down = max(w_gate.shape[1], 1), max(w_down.shape[1], 1)
    st = _lib.dgemm_gated_ffn_backward(
        dt, act, OP_T if trans_w else OP_N, M, D, F, dy.data_ptr(), lddy, x.data_ptr(), ldx,
        w_gate.data_ptr(), ldwg, w_up.data_ptr(), ldwu, w_down.data_ptr(), ldwd, g.data_ptr(), ldg,
        u.data_ptr(), ldu, h.data_ptr(), ldh, dg.data_ptr(), lddg, du.data_ptr(), lddu,
        dx.data_ptr(), max(D, 1), dwg.data_ptr(), up, dwu.data_ptr(), up, dwd.data_ptr(), down,
        handle)
    _check(st, "gated_ffn_backward")
    return dx, dwg, dwu, dwd
