"""The feed-forward operators over torch CUDA tensors: layer norm, the linear
layer with bias, activation and residual in its epilogue, and the gated
feed-forward block, each with its backward pass; the two products with weights in
8-bit integers; and the orthogonalised update of a weight.

Like `matmul`, these only check shapes and types, derive pointers, leading
dimensions and the stream, allocate outputs and workspaces, and raise on a
non-zero status (csrc/torch_binding.cpp, built beside libdgemm.so); all
arithmetic runs in the library's kernels.  Activations may have any number of
leading dimensions that flatten into rows without a copy; the last dimension
is contiguous.  Outputs are allocated on the stream the call runs on
(`stream`: a torch.cuda.Stream or raw handle, default the current one); tensors
made on another stream must be ready there, as for any torch call.  Shapes and
types that do not fit raise ValueError and TypeError before anything runs.

Autograd records nothing of these calls: with gradients enabled, layer_norm,
linear and gated_ffn refuse arguments that require them (RuntimeError); call them
under torch.no_grad() and the `_backward` calls for the gradients.
"""
import importlib.machinery
import importlib.util
import os

from . import _lib
from ._lib import ACT_GELU, ACT_GELU_TANH, ACT_NONE, ACT_RELU, ACT_SILU, LibraryMissing

ACTIVATIONS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH,
               "silu": ACT_SILU}

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_torch_binding.so")

_binding = None


def _raise(status, what):
    from . import DgemmError

    raise DgemmError(status, what)


def _load():
    """Load _torch_binding.so (built by dense_gemm_f32_gb300.build); raise if it is absent or
    was built for another PyTorch or Python."""
    global _binding
    if _binding is None:
        import torch  # noqa: F401  (the libraries that the module links to)

        _lib.load()  # the same libdgemm.so serves both
        if not os.path.exists(BINDING_PATH):
            raise LibraryMissing(
                f"{BINDING_PATH} is missing: build it first with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        from . import build

        if build.built_key(BINDING_PATH) != build.binding_key():
            raise LibraryMissing(
                f"{BINDING_PATH} was built for {build.built_key(BINDING_PATH)}, this is "
                f"{build.binding_key()}: build it again with "
                "`python -c 'import __graft_entry__ as g; g.build()'`")
        name = "_torch_binding"
        loader = importlib.machinery.ExtensionFileLoader(name, BINDING_PATH)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_file_location(name, BINDING_PATH, loader=loader))
        loader.exec_module(module)
        module.on_error(_raise)
        _binding = module
    return _binding


def _on(stream, x):
    """The given stream (object or raw handle) as a context."""
    import torch

    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream, device=x.device)
    return torch.cuda.stream(stream)


def _activation(name):
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)}, got {name!r}")
    return code


def layer_norm(x, weight=None, bias=None, eps=1e-5, return_stats=False, out=None, stream=None):
    """y = (x - mean) rstd weight + bias over the last dimension.

    x: (..., n) bfloat16, float16 or float32.  weight, bias: n elements of the
    same type, or None.  out: optional tensor of x's shape and type to write.
    Returns y, or (y, mean, rstd) with the float32 statistics of every row
    (shape x.shape[:-1]) that layer_norm_backward takes; rows without columns
    have none (NaN).
    """
    if stream is not None:
        with _on(stream, x):
            return layer_norm(x, weight, bias, eps, return_stats, out)
    return (_binding or _load()).layer_norm(x, weight, bias, eps, return_stats, out)


def layer_norm_backward(dy, x, weight, mean, rstd, dresidual=None, stream=None):
    """(dx, dweight, dbias) of layer_norm.

    mean, rstd: what layer_norm returned.  dresidual: a gradient of x's shape
    that joins dx (that of a skip connection around the norm), or None.  weight
    may be None (then 1; dweight is still returned).
    """
    if stream is not None:
        with _on(stream, x):
            return layer_norm_backward(dy, x, weight, mean, rstd, dresidual)
    return (_binding or _load()).layer_norm_backward(dy, x, weight, mean, rstd, dresidual)


def linear(x, w, bias=None, activation="none", residual=None, trans_w=False, return_preact=False,
           out=None, stream=None):
    """act(x @ op(w) + bias) + residual in one kernel.

    x: (..., K) bfloat16 or float16; w: K x N, or N x K with trans_w; bias: N
    elements; residual: (..., N); all of x's type.  out: optional (..., N)
    tensor to write, which may be `residual` itself.  Returns d, or
    (d, preact) with preact = x @ op(w) + bias, which linear_backward takes.
    """
    if stream is not None:
        with _on(stream, x):
            return linear(x, w, bias, activation, residual, trans_w, return_preact, out)
    return (_binding or _load()).linear(x, w, bias, _activation(activation), residual, trans_w,
                                        return_preact, out)


def linear_backward(dd, x, w, activation="none", preact=None, trans_w=False, with_bias=True,
                    stream=None):
    """(dx, dw, dbias) of linear; dbias is None without with_bias.

    dd: the gradient of linear's result (also that of its residual).  preact:
    what linear(..., return_preact=True) returned; needed unless activation is
    "none".  dd act'(preact) is rounded to x's type before the two products (in
    float16 it is infinite past 65504); dbias sums the values before that.
    """
    if stream is not None:
        with _on(stream, x):
            return linear_backward(dd, x, w, activation, preact, trans_w, with_bias)
    return (_binding or _load()).linear_backward(dd, x, w, _activation(activation), preact, trans_w,
                                                 with_bias)


def gated_ffn(x, w_gate, w_up, w_down, activation="silu", residual=None, trans_w=False,
              return_saved=False, out=None, stream=None):
    """(act(x @ op(w_gate)) * (x @ op(w_up))) @ op(w_down) + residual.

    x: (..., D) bfloat16 or float16.  w_gate, w_up: D x F and w_down: F x D, or
    their transposes with trans_w.  residual: of x's shape; out may be it.
    Returns y, or (y, g, u) with the two projections, (..., F), which
    gated_ffn_backward takes.  The hidden units are computed in float32 and
    rounded to x's type for the product with w_down (in float16 they are
    infinite past 65504).
    """
    if stream is not None:
        with _on(stream, x):
            return gated_ffn(x, w_gate, w_up, w_down, activation, residual, trans_w, return_saved,
                             out)
    return (_binding or _load()).gated_ffn(x, w_gate, w_up, w_down, _activation(activation),
                                           residual, trans_w, return_saved, out)


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, g, u, activation="silu", trans_w=False,
                       stream=None):
    """(dx, dw_gate, dw_up, dw_down) of gated_ffn from its saved g and u.

    dy: the gradient of gated_ffn's result (also that of its residual).  The
    gradients of g and u, and the hidden units computed again from them, are
    rounded to x's type before the products that read them (in float16 they are
    infinite past 65504).
    """
    if stream is not None:
        with _on(stream, x):
            return gated_ffn_backward(dy, x, w_gate, w_up, w_down, g, u, activation, trans_w)
    return (_binding or _load()).gated_ffn_backward(dy, x, w_gate, w_up, w_down, g, u,
                                                    _activation(activation), trans_w)


def quantize_int8(x, transpose=False, stream=None):
    """(q, scale): every row of x as 8-bit integers, x about q * scale[..., None].

    x: (..., n) bfloat16, float16 or float32.  q: int8 of x's shape, at most 127
    in size, round(127 x / max|x|) with ties to even; scale: float32, max|x| / 127
    of every row (shape x.shape[:-1]).  transpose: x is a K x N matrix whose
    columns are meant: q is N x K and scale has N elements, the form in which
    linear_int8 and gated_ffn_int8 take weights that linear and gated_ffn have as
    K x N.  A row with NaN or an infinity gets that for its scale, and zeros.  The rows
    of q start on 16-byte boundaries, as the products read weights best (so q is
    contiguous where they are a multiple of 16 long; other weights are copied first, in
    every call).
    """
    if stream is not None:
        with _on(stream, x):
            return quantize_int8(x, transpose)
    return (_binding or _load()).quantize_int8(x, transpose)


def linear_int8(x, w, w_scale, bias=None, activation="none", residual=None, x_scale=None, dtype=None,
                out=None, stream=None):
    """act(x @ (w * w_scale[:, None]).T + bias) + residual, multiplied in 8-bit integers.

    w: N x K int8 and w_scale: N float32, as quantize_int8 gives them (w.T of what
    linear takes).  x: (..., K) bfloat16 or float16, put into 8 bits in the call,
    each row with a scale of its own; or int8 with x_scale, float32 of shape
    x.shape[:-1], to use the integers for several products.  bias: N elements;
    residual, and out if given (it may be `residual` itself): (..., N); all of the
    result's type, which is x's, or for an int8 x `dtype` (default bfloat16).
    Sums of integers are exact within 2^24 and rounded to float32 beyond.
    """
    if stream is not None:
        with _on(stream, x):
            return linear_int8(x, w, w_scale, bias, activation, residual, x_scale, dtype, out)
    return (_binding or _load()).linear_int8(x, w, w_scale, bias, _activation(activation), residual,
                                             x_scale, dtype, out)


def gated_ffn_int8(x, w_gate, gate_scale, w_up, up_scale, w_down, down_scale, activation="silu",
                   residual=None, out=None, stream=None):
    """gated_ffn with its weights, and the rows they multiply, in 8-bit integers.

    x: (..., D) bfloat16 or float16.  w_gate, w_up: F x D and w_down: D x F int8,
    with the float32 scales of their rows, as quantize_int8 gives them.  residual:
    of x's shape; out may be it.  The hidden units are float32 until they are put
    into 8 bits, each row with a scale of its own.
    """
    if stream is not None:
        with _on(stream, x):
            return gated_ffn_int8(x, w_gate, gate_scale, w_up, up_scale, w_down, down_scale,
                                  activation, residual, out)
    return (_binding or _load()).gated_ffn_int8(x, w_gate, gate_scale, w_up, up_scale, w_down,
                                                down_scale, _activation(activation), residual, out)


def orthogonalize(x, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=1.0, residual=None,
                  residual_scale=1.0, out=None, stream=None):
    """scale * orthogonalised(x) + residual_scale * residual, x's singular values brought towards 1
    by `steps` Newton-Schulz steps (the Muon optimiser's update of a weight matrix):

        x0 = x / (|x| + eps);  x <- a x + (b A + c A A) x,  A = x x^T.

    x: a 2-D matrix, bfloat16, float16 or float32 (a momentum).  coefficients: (a, b,
    c), or a sequence of `steps` such triples.  residual (the weights) and out: x's shape
    and either of these types; out may be residual itself; the result has residual's type,
    else out's, else x's.  So orthogonalize(m, scale=-lr, residual=w,
    residual_scale=1 - lr * decay, out=w) is a step of the optimiser.  The products
    are fp16 with float32 sums, whatever the types (a float32 x begins as two fp16 terms): five steps are off by some 0.0015 of the
    update's norm for a usual gradient, up to 0.008 where the singular values fall steeply, and
    at most 0.02 (a matrix of rank one; 0.07 with 2 to 7 rows or columns); more steps enlarge what
    was rounded.
    """
    if stream is not None:
        with _on(stream, x):
            return orthogonalize(x, steps, coefficients, eps, scale, residual, residual_scale, out)
    return (_binding or _load()).orthogonalize(x, steps, coefficients, eps, scale, residual,
                                               residual_scale, out)
