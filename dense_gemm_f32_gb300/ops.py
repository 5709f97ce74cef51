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

A small call is over in a few microseconds on the GPU, so what runs here is
kept short: no closures or views on the way, and the current stream's handle
without the stream object (12 against 25 us for layer_norm of one 4096-wide
row with its statistics on a GB300's host).
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
_empty, _empty_like = torch.empty, torch.empty_like


def _raise(status, what):
    from . import DgemmError

    raise DgemmError(status, what)


def _current(x):
    """The raw handle of the current stream of x's device."""
    if not x.is_cuda:
        raise ValueError("expected CUDA tensors")
    return torch._C._cuda_getCurrentRawStream(x.get_device())


def _on(stream, x):
    """The given stream (object or raw handle) as a torch stream."""
    if hasattr(stream, "cuda_stream"):
        return stream
    return torch.cuda.ExternalStream(stream, device=x.device)


def _code(table, name, x):
    code = table.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} takes {', '.join(str(d) for d in table)}, got {x.dtype}")
    return code


def _rows(x, name, dtype, cols=None):
    """(rows, cols, leading dimension) of x with its leading dimensions flattened."""
    if x.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {x.dtype}")
    if x.dim() != 2:
        if x.dim() == 0:
            raise ValueError(f"{name}: expected at least one dimension")
        c = x.shape[-1]
        try:
            x = x.view(x.shape[:-1].numel(), c)
        except RuntimeError:
            raise ValueError(f"{name}: the leading dimensions do not flatten into rows") from None
    r, c = x.shape
    ld, inner = x.stride()
    if cols is not None and c != cols:
        raise ValueError(f"{name}: the last dimension is {c}, expected {cols}")
    if inner != 1 and c > 1 and r > 0:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return r, c, ld if r > 1 else c or 1


def _like(x, name, dtype, rows, cols):
    """Leading dimension of x, which has to be rows x cols."""
    r, _, ld = _rows(x, name, dtype, cols)
    if r != rows:
        raise ValueError(f"{name}: {r} rows, expected {rows}")
    return ld


def _optional(x, name, dtype, rows, cols):
    """(pointer, leading dimension) of an optional matrix."""
    if x is None:
        return 0, cols or 1
    return x.data_ptr(), _like(x, name, dtype, rows, cols)


def _vector(x, name, dtype, n):
    if x is None:
        return 0
    if x.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {x.dtype}")
    if x.dim() != 1 or x.shape[0] != n:
        raise ValueError(f"{name}: expected {n} elements, got {tuple(x.shape)}")
    if n > 1 and x.stride(0) != 1:
        raise ValueError(f"{name}: must be contiguous")
    return x.data_ptr()


def _weight(w, name, dtype, inner, outer, trans_w):
    """Leading dimension of a weight: inner x outer, or outer x inner when trans_w."""
    rows, cols = (outer, inner) if trans_w else (inner, outer)
    if w.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {w.dtype}")
    if tuple(w.shape) != (rows, cols):
        raise ValueError(f"{name}: expected {rows}x{cols}, got {tuple(w.shape)}")
    return _rows(w, name, dtype)[2]


def _activation(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)}, got {name!r}")
    return code


def _new(x):
    """An uninitialised contiguous tensor like x."""
    return _empty_like(x) if x.is_contiguous() else _empty(x.shape, dtype=x.dtype, device=x.device)


def _pitched(rows, cols, like):
    """A rows x cols workspace whose rows start on 16-byte boundaries, and its pitch."""
    ld = (cols + 7) // 8 * 8
    return _empty((rows, ld), dtype=like.dtype, device=like.device), ld or 1


def layer_norm(x, weight=None, bias=None, eps=1e-5, return_stats=False, out=None, stream=None):
    """y = (x - mean) rstd weight + bias over the last dimension.

    x: (..., n) bfloat16, float16 or float32.  weight, bias: n elements of the
    same type, or None.  out: optional tensor of x's shape and type to write.
    Returns y, or (y, mean, rstd) with the float32 statistics of every row
    (shape x.shape[:-1]) that layer_norm_backward takes.
    """
    if stream is not None:
        with torch.cuda.stream(_on(stream, x)):
            return layer_norm(x, weight, bias, eps, return_stats, out)
    dtype = x.dtype
    dt = _code(_FLOAT, "layer_norm", x)
    rows, cols, ldx = _rows(x, "x", dtype)
    pw, pb = _vector(weight, "weight", dtype, cols), _vector(bias, "bias", dtype, cols)
    if out is None:
        y, ldy = _new(x), cols or 1
    else:
        if out.shape != x.shape:
            raise ValueError(f"out: expected {tuple(x.shape)}, got {tuple(out.shape)}")
        y, ldy = out, _like(out, "out", dtype, rows, cols)
    handle = _current(x)
    if return_stats:
        shape = (rows,) if x.dim() == 2 else x.shape[:-1]
        mean = _empty(shape, dtype=torch.float32, device=x.device)
        rstd = _empty(shape, dtype=torch.float32, device=x.device)
        pm, ps = mean.data_ptr(), rstd.data_ptr()
    else:
        pm = ps = 0
    st = _lib.load().dgemm_layer_norm(dt, rows, cols, eps, x.data_ptr(), ldx, pw, pb, y.data_ptr(),
                                      ldy, pm, ps, handle)
    if st != OK:
        _raise(st, "layer_norm")
    return (y, mean, rstd) if return_stats else y


def layer_norm_backward(dy, x, weight, mean, rstd, dresidual=None, stream=None):
    """(dx, dweight, dbias) of layer_norm.

    mean, rstd: what layer_norm returned.  dresidual: a gradient of x's shape
    that joins dx (that of a skip connection around the norm), or None.  weight
    may be None (then 1; dweight is still returned).
    """
    if stream is not None:
        with torch.cuda.stream(_on(stream, x)):
            return layer_norm_backward(dy, x, weight, mean, rstd, dresidual)
    dtype = x.dtype
    dt = _code(_FLOAT, "layer_norm_backward", x)
    rows, cols, ldx = _rows(x, "x", dtype)
    lddy = _like(dy, "dy", dtype, rows, cols)
    pr, lddr = _optional(dresidual, "dresidual", dtype, rows, cols)
    pw = _vector(weight, "weight", dtype, cols)
    pm = _vector(mean if mean.dim() == 1 else mean.reshape(-1), "mean", torch.float32, rows)
    ps = _vector(rstd if rstd.dim() == 1 else rstd.reshape(-1), "rstd", torch.float32, rows)
    handle = _current(x)
    dx = _new(x)
    dw = _empty((cols,), dtype=dtype, device=x.device)
    db = _empty_like(dw)
    st = _lib.load().dgemm_layer_norm_backward(dt, rows, cols, dy.data_ptr(), lddy, x.data_ptr(),
                                               ldx, pw, pm, ps, pr, lddr, dx.data_ptr(), cols or 1,
                                               dw.data_ptr(), db.data_ptr(), handle)
    if st != OK:
        _raise(st, "layer_norm_backward")
    return dx, dw, db


def _layer(what, x, w, trans_w):
    """Type code, sizes and leading dimensions of a linear layer's input and weight."""
    dt = _code(_HALF, what, x)
    if w.dim() != 2:
        raise ValueError("w: expected a 2-D matrix")
    M, K, ldx = _rows(x, "x", x.dtype)
    N = w.shape[0] if trans_w else w.shape[1]
    return dt, M, N, K, ldx, _weight(w, "w", x.dtype, K, N, trans_w)


def linear(x, w, bias=None, activation="none", residual=None, trans_w=False, return_preact=False,
           out=None, stream=None):
    """act(x @ op(w) + bias) + residual in one kernel.

    x: (..., K) bfloat16 or float16; w: K x N, or N x K with trans_w; bias: N
    elements; residual: (..., N); all of x's type.  out: optional (..., N)
    tensor to write, which may be `residual` itself.  Returns d, or
    (d, preact) with preact = x @ op(w) + bias, which linear_backward takes.
    """
    if stream is not None:
        with torch.cuda.stream(_on(stream, x)):
            return linear(x, w, bias, activation, residual, trans_w, return_preact, out)
    act = _activation(activation)
    dt, M, N, K, ldx, ldw = _layer("linear", x, w, trans_w)
    dtype = x.dtype
    pb = _vector(bias, "bias", dtype, N)
    pr, ldr = _optional(residual, "residual", dtype, M, N)
    shape = (M, N) if x.dim() == 2 else x.shape[:-1] + (N,)
    if out is not None and tuple(out.shape) != tuple(shape):
        raise ValueError(f"out: expected {tuple(shape)}, got {tuple(out.shape)}")
    handle = _current(x)
    if out is None:
        d, ldd = _empty(shape, dtype=dtype, device=x.device), N or 1
    else:
        d, ldd = out, _like(out, "out", dtype, M, N)
    z = _empty(shape, dtype=dtype, device=x.device) if return_preact else None
    st = _lib.load().dgemm_linear(dt, act, OP_T if trans_w else OP_N, M, N, K, x.data_ptr(), ldx,
                                  w.data_ptr(), ldw, pb, pr, ldr, d.data_ptr(), ldd,
                                  z.data_ptr() if return_preact else 0, N or 1, handle)
    if st != OK:
        _raise(st, "linear")
    return (d, z) if return_preact else d


def linear_backward(dd, x, w, activation="none", preact=None, trans_w=False, with_bias=True,
                    stream=None):
    """(dx, dw, dbias) of linear; dbias is None without with_bias.

    dd: the gradient of linear's result (also that of its residual).  preact:
    what linear(..., return_preact=True) returned; needed unless activation is
    "none".
    """
    if stream is not None:
        with torch.cuda.stream(_on(stream, x)):
            return linear_backward(dd, x, w, activation, preact, trans_w, with_bias)
    act = _activation(activation)
    dt, M, N, K, ldx, ldw = _layer("linear_backward", x, w, trans_w)
    dtype = x.dtype
    lddd = _like(dd, "dd", dtype, M, N)
    if act == ACT_NONE:
        pz, ldz, dz, pdz, lddz = 0, N or 1, None, 0, N or 1
    else:
        if preact is None:
            raise ValueError(f"preact is needed for activation {activation!r}")
        pz, ldz = preact.data_ptr(), _like(preact, "preact", dtype, M, N)
        dz, lddz = _pitched(M, N, x)
        pdz = dz.data_ptr()
    handle = _current(x)
    dx, dw = _new(x), _new(w)
    db = _empty((N,), dtype=dtype, device=x.device) if with_bias else None
    st = _lib.load().dgemm_linear_backward(dt, act, OP_T if trans_w else OP_N, M, N, K,
                                           dd.data_ptr(), lddd, x.data_ptr(), ldx, w.data_ptr(),
                                           ldw, pz, ldz, pdz, lddz, dx.data_ptr(), K or 1,
                                           dw.data_ptr(), w.shape[1] or 1,
                                           db.data_ptr() if with_bias else 0, handle)
    if st != OK:
        _raise(st, "linear_backward")
    return dx, dw, db


def _block(what, x, w_gate, w_up, w_down, trans_w):
    """Type code, sizes and leading dimensions of a gated block's input and weights."""
    dt = _code(_HALF, what, x)
    dtype = x.dtype
    if w_gate.dim() != 2:
        raise ValueError("w_gate: expected a 2-D matrix")
    M, D, ldx = _rows(x, "x", dtype)
    F = w_gate.shape[0] if trans_w else w_gate.shape[1]
    return (dt, M, D, F, ldx, _weight(w_gate, "w_gate", dtype, D, F, trans_w),
            _weight(w_up, "w_up", dtype, D, F, trans_w),
            _weight(w_down, "w_down", dtype, F, D, trans_w))


def gated_ffn(x, w_gate, w_up, w_down, activation="silu", residual=None, trans_w=False,
              return_saved=False, out=None, stream=None):
    """(act(x @ op(w_gate)) * (x @ op(w_up))) @ op(w_down) + residual.

    x: (..., D) bfloat16 or float16.  w_gate, w_up: D x F and w_down: F x D, or
    their transposes with trans_w.  residual: of x's shape; out may be it.
    Returns y, or (y, g, u) with the two projections, (..., F), which
    gated_ffn_backward takes.
    """
    if stream is not None:
        with torch.cuda.stream(_on(stream, x)):
            return gated_ffn(x, w_gate, w_up, w_down, activation, residual, trans_w, return_saved,
                             out)
    act = _activation(activation)
    dt, M, D, F, ldx, ldwg, ldwu, ldwd = _block("gated_ffn", x, w_gate, w_up, w_down, trans_w)
    dtype = x.dtype
    pr, ldr = _optional(residual, "residual", dtype, M, D)
    if out is not None and out.shape != x.shape:
        raise ValueError(f"out: expected {tuple(x.shape)}, got {tuple(out.shape)}")
    handle = _current(x)
    if out is None:
        y, ldy = _new(x), D or 1
    else:
        y, ldy = out, _like(out, "out", dtype, M, D)
    g = u = None
    pg = pu = 0
    if return_saved:
        shape = (M, F) if x.dim() == 2 else x.shape[:-1] + (F,)
        g = _empty(shape, dtype=dtype, device=x.device)
        u = _empty_like(g)
        pg, pu = g.data_ptr(), u.data_ptr()
    h, ldh = _pitched(M, F, x)
    st = _lib.load().dgemm_gated_ffn(dt, act, OP_T if trans_w else OP_N, M, D, F, x.data_ptr(), ldx,
                                     w_gate.data_ptr(), ldwg, w_up.data_ptr(), ldwu,
                                     w_down.data_ptr(), ldwd, pr, ldr, h.data_ptr(), ldh, pg,
                                     F or 1, pu, F or 1, y.data_ptr(), ldy, handle)
    if st != OK:
        _raise(st, "gated_ffn")
    return (y, g, u) if return_saved else y


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, g, u, activation="silu", trans_w=False,
                       stream=None):
    """(dx, dw_gate, dw_up, dw_down) of gated_ffn from its saved g and u.

    dy: the gradient of gated_ffn's result (also that of its residual).
    """
    if stream is not None:
        with torch.cuda.stream(_on(stream, x)):
            return gated_ffn_backward(dy, x, w_gate, w_up, w_down, g, u, activation, trans_w)
    act = _activation(activation)
    dt, M, D, F, ldx, ldwg, ldwu, ldwd = _block("gated_ffn_backward", x, w_gate, w_up, w_down,
                                                trans_w)
    dtype = x.dtype
    lddy = _like(dy, "dy", dtype, M, D)
    ldg, ldu = _like(g, "g", dtype, M, F), _like(u, "u", dtype, M, F)
    handle = _current(x)
    dx, dwg, dwu, dwd = _new(x), _new(w_gate), _new(w_up), _new(w_down)
    h, ldh = _pitched(M, F, x)
    dg, du = _empty_like(h), _empty_like(h)
    up, down = w_gate.shape[1] or 1, w_down.shape[1] or 1
    st = _lib.load().dgemm_gated_ffn_backward(
        dt, act, OP_T if trans_w else OP_N, M, D, F, dy.data_ptr(), lddy, x.data_ptr(), ldx,
        w_gate.data_ptr(), ldwg, w_up.data_ptr(), ldwu, w_down.data_ptr(), ldwd, g.data_ptr(), ldg,
        u.data_ptr(), ldu, h.data_ptr(), ldh, dg.data_ptr(), ldh, du.data_ptr(), ldh,
        dx.data_ptr(), D or 1, dwg.data_ptr(), up, dwu.data_ptr(), up, dwd.data_ptr(), down,
        handle)
    if st != OK:
        _raise(st, "gated_ffn_backward")
    return dx, dwg, dwu, dwd
