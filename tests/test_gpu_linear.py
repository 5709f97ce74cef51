"""The linear layer on the GPU, forward and backward, against the 64-bit
reference within bounds derived in ops_reference.py."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import ops_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]
# (M, N, K): one token, a few, around tile edges, odd everywhere, K of one
# element up to many tiles, N of one column
SHAPES = [(1, 64, 64), (1, 1000, 4096), (2, 8, 1), (3, 1, 17), (16, 136, 520), (17, 129, 65),
          (64, 512, 2048), (100, 257, 1000), (128, 128, 128), (129, 300, 72), (255, 96, 333),
          (257, 512, 64), (1000, 1013, 997), (700, 2048, 256), (2100, 1032, 130)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def _d(t):
    return None if t is None else t.double()


def _layer(M, N, K, dtype, seed, bias=True, residual=True):
    n = ref.make(seed)
    x, w = n((M, K), dtype), n((K, N), dtype, max(K, 1) ** -0.5)
    return (n, x, w, n((N,), dtype, 0.5) if bias else None,
            n((M, N), dtype) if residual else None)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("M, N, K", SHAPES)
def test_forward(M, N, K, trans_w, dtype):
    act = ref.ACTS[(M + N + K) % 5]
    _, x, w, b, r = _layer(M, N, K, dtype, M + N + K)
    ws = w.t().contiguous() if trans_w else w
    d, z = dg.linear(x, ws, b, act, r, trans_w=trans_w, return_preact=True)
    want = ref.linear(_d(x), _d(w), _d(b), act, _d(r), dtype)
    ref.check(d, want[0], f"d {act}")
    ref.check(z, want[1], "z")
    assert torch.equal(dg.linear(x, ws, b, act, r, trans_w=trans_w), d)
    gu.check_watchdog()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("act", ref.ACTS)
def test_every_activation_with_and_without_bias_and_residual(act, M, dtype):
    for bias in (False, True):
        for residual in (False, True):
            _, x, w, b, r = _layer(M, 200, 104, dtype, 7, bias, residual)
            x = x * 3  # out to where the activations saturate
            got = dg.linear(x, w, b, act, r)
            ref.check(got, ref.linear(_d(x), _d(w), _d(b), act, _d(r), dtype)[0],
                      f"{act} bias {bias} residual {residual}")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("M, N, K", SHAPES)
def test_backward(M, N, K, trans_w, dtype):
    act = ref.ACTS[(M + N + 2 * K) % 5]
    n, x, w, b, _ = _layer(M, N, K, dtype, M + N + K, residual=False)
    ws = w.t().contiguous() if trans_w else w
    dd = n((M, N), dtype, 0.2)
    _, z = dg.linear(x, ws, b, act, trans_w=trans_w, return_preact=True)
    got = dg.linear_backward(dd, x, ws, act, z, trans_w=trans_w)
    want = ref.linear_backward(_d(dd), _d(x), _d(w), act, _d(z), dtype)
    for g, w_, what in zip((got[0], got[1].t() if trans_w else got[1], got[2]), want,
                           ("dx", "dw", "dbias")):
        ref.check(g, w_, f"{what} {act}")
    assert dg.linear_backward(dd, x, ws, act, z, trans_w=trans_w, with_bias=False)[2] is None
    again = dg.linear_backward(dd, x, ws, act, z, trans_w=trans_w)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    gu.check_watchdog()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M, N, K", [(3, 72, 80), (70, 130, 200), (600, 520, 136)])
@pytest.mark.parametrize("pad, offset", [(0, 8), (8, 0), (3, 1), (1, 0)])
def test_strides_alignment_and_guards(M, N, K, pad, offset, dtype):
    """Operands, residual and outputs in wider buffers, aligned or not; the
    gaps of the outputs stay as they were."""
    n, x, w, b, r = _layer(M, N, K, dtype, 5)
    xs, ws, rs = (ref.pitched(t, t.shape[1] + pad, offset) for t in (x, w, r))
    bs = ref.pitched(b[None], N, offset)[0]
    buf = torch.full((offset + M * (N + pad) + 64,), 7.0, dtype=dtype, device="cuda")
    out = buf.as_strided((M, N), (N + pad, 1), offset)
    want, wz = ref.linear(_d(x), _d(w), _d(b), "gelu", _d(r), dtype)
    dg.linear(xs, ws, bs, "gelu", rs, out=out)
    ref.check(out, want, "d")
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep.as_strided((M, N), (N + pad, 1), offset).fill_(False)
    assert (buf[keep] == 7.0).all()
    _, z = dg.linear(xs, ws, bs, "gelu", return_preact=True)
    ref.check(z, wz, "z")
    dd = n((M, N), dtype, 0.2)
    got = dg.linear_backward(ref.pitched(dd, N + pad, offset), xs, ws, "gelu",
                             ref.pitched(z, N + pad, offset))
    for g, w_, what in zip(got, ref.linear_backward(_d(dd), _d(x), _d(w), "gelu", _d(z), dtype),
                           ("dx", "dw", "dbias")):
        ref.check(g, w_, what)


@pytest.mark.parametrize("M", [2, 400])
def test_residual_in_place(M):
    _, x, w, b, r = _layer(M, 264, 128, torch.bfloat16, 3)
    want = dg.linear(x, w, b, "silu", r)
    out = dg.linear(x, w, b, "silu", r, out=r)
    assert out is r and torch.equal(r, want)


def test_empty_sums_and_empty_shapes():
    _, x, w, b, r = _layer(5, 40, 0, torch.float16, 1)
    got = dg.linear(x, w, b, "gelu", r)  # K = 0: act(bias) + residual
    ref.check(got, ref.linear(_d(x), _d(w), _d(b), "gelu", _d(r), torch.float16)[0], "K = 0")
    _, x, w, b, r = _layer(300, 300, 0, torch.float16, 1)
    ref.check(dg.linear(x, w, b, "gelu", r),
              ref.linear(_d(x), _d(w), _d(b), "gelu", _d(r), torch.float16)[0], "K = 0, many tiles")
    _, x, w, _, _ = _layer(0, 40, 24, torch.float16, 1)
    assert dg.linear(x, w).shape == (0, 40)
    dx, dw, db = dg.linear_backward(x[:, :0].new_zeros((0, 40)), x, w)
    assert dx.shape == (0, 24) and not dw.any() and not db.any()
    _, x, w, _, _ = _layer(6, 0, 24, torch.float16, 1)
    assert dg.linear(x, w).shape == (6, 0)
    dx, dw, db = dg.linear_backward(x.new_zeros((6, 0)), x, w)
    assert not dx.any() and dw.shape == (24, 0) and db.shape == (0,)


def test_leading_dimensions_and_streams():
    _, x, w, b, r = _layer(24, 72, 40, torch.bfloat16, 2)
    want = dg.linear(x, w, b, "relu", r)
    assert torch.equal(dg.linear(x.view(2, 3, 4, 40), w, b, "relu", r.view(2, 3, 4, 72)),
                       want.view(2, 3, 4, 72))
    assert torch.equal(dg.linear(x[0], w, b, "relu", r[0]), want[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        got = dg.linear(x, w, b, "relu", r, stream=stream)
        s.synchronize()
        assert torch.equal(got, want)


def test_special_values_stay_where_the_formula_puts_them():
    """Zero rows give act(bias); an infinity or NaN in one row of x reaches that row only."""
    _, x, w, b, _ = _layer(200, 136, 64, torch.bfloat16, 8, residual=False)
    x[0] = 0
    x[3, 5] = float("inf")
    x[7, 63] = float("nan")
    d = dg.linear(x, w, b, "relu")
    assert torch.equal(d[0], b.clamp(min=0))
    assert torch.isnan(d[7]).all() and not torch.isfinite(d[3]).all()
    rest = [i for i in range(200) if i not in (3, 7)]
    assert torch.isfinite(d[rest]).all()


def test_large_offsets():
    """Rows more than 2^32 elements into their buffers."""
    M, N, K, ld = 40, 48, 32, 1 << 27
    _, x, w, b, r = _layer(M, N, K, torch.float16, 6)
    want = dg.linear(x, w, b, "silu", r)
    buf = torch.zeros(M * ld, dtype=torch.float16, device="cuda")
    xs, rs = buf.as_strided((M, K), (ld, 1), 0), buf.as_strided((M, N), (ld, 1), 64)
    out = buf.as_strided((M, N), (ld, 1), 256)
    xs.copy_(x), rs.copy_(r)
    # the windows interleave: an output inside an input's span is refused
    with pytest.raises(dg.DgemmError):
        dg.linear(xs, w, b, "silu", rs, out=out)
    assert torch.equal(dg.linear(xs, w, b, "silu", rs), want)


def test_gradients_against_differences():
    """<grad, v> against central differences of the 64-bit forward form, within
    the roundings of dz and of the stored gradient."""
    n, x, w, b, _ = _layer(20, 48, 32, torch.float16, 4, residual=False)
    c = n((20, 48), torch.float16)
    z = ref.linear(_d(x), _d(w), _d(b), "gelu_tanh", None, torch.float16)[1][0].half()
    got = dg.linear_backward(c, x, w, "gelu_tanh", z)
    f = lambda *t: (_d(c) * ref.linear(*t, "gelu_tanh", None, torch.float16)[0][0]).sum()  # noqa: E731
    h = 1e-5
    for i, t in enumerate((x, w, b)):
        v = n(t.shape, torch.float32).double()
        up, down = [_d(x), _d(w), _d(b)], [_d(x), _d(w), _d(b)]
        up[i], down[i] = _d(t) + h * v, _d(t) - h * v
        want = (f(*up) - f(*down)) / (2 * h)
        # z (rounded), dz and the gradient round by 2^-11 each: 2^-9 of sum |grad v|
        # for the gradient itself, and sqrt-sized sums of the others stay below it
        assert abs((_d(got[i]) * v).sum() - want) <= 2.0 ** -9 * (_d(got[i]) * v).abs().sum()
