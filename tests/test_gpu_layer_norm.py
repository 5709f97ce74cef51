"""Layer norm on the GPU, forward and backward, against the 64-bit reference
within bounds derived in ops_reference.py."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import ops_reference as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# one row, one column, sizes around a warp's and a block's share, odd sizes,
# rows longer than a block keeps in registers
SHAPES = [(1, 1), (1, 4096), (3, 2), (5, 31), (17, 64), (2, 1000), (1000, 1013), (33, 1024),
          (7, 1025), (300, 4096), (129, 8200), (3, 16384), (2, 40001), (2, 70000), (5000, 72)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def _inputs(rows, cols, dtype, seed):
    n = ref.make(seed)
    x = n((rows, cols), dtype, 1.5, 0.25)
    if cols > 8:
        x[:, cols // 3] *= 20.0
    return n, x, n((cols,), dtype, 0.2, 1.0), n((cols,), dtype, 0.2)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_forward(rows, cols, dtype):
    _, x, w, b = _inputs(rows, cols, dtype, rows + cols)
    y, mean, rstd = dg.layer_norm(x, w, b, eps=EPS, return_stats=True)
    want = ref.layer_norm(x.double(), w.double(), b.double(), EPS, dtype)
    for got, w_, what in zip((y, mean, rstd), want, ("y", "mean", "rstd")):
        ref.check(got, w_, f"{what} {rows}x{cols} {dtype}")
    assert torch.equal(dg.layer_norm(x, w, b, eps=EPS), y)  # the same bits without statistics


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows, cols", SHAPES)
@pytest.mark.parametrize("skip", [False, True])
def test_backward(rows, cols, dtype, skip):
    n, x, w, _ = _inputs(rows, cols, dtype, rows * 3 + cols)
    dy = n((rows, cols), dtype, 0.1)
    dr = n((rows, cols), dtype, 0.1) if skip else None
    _, mean, rstd = dg.layer_norm(x, w, None, eps=EPS, return_stats=True)
    got = dg.layer_norm_backward(dy, x, w, mean, rstd, dresidual=dr)
    want = ref.layer_norm_backward(dy.double(), x.double(), w.double(), mean.double(),
                                   rstd.double(), None if dr is None else dr.double(), dtype)
    for g, w_, what in zip(got, want, ("dx", "dweight", "dbias")):
        ref.check(g, w_, f"{what} {rows}x{cols} {dtype}")
    again = dg.layer_norm_backward(dy, x, w, mean, rstd, dresidual=dr)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_strided_rows_odd_offsets_and_no_parameters(dtype):
    n, x, w, b = _inputs(37, 201, dtype, 4)
    dy = n((37, 201), dtype, 0.1)
    for ld, off in ((208, 0), (203, 1), (216, 3)):
        xs, dys = ref.pitched(x, ld, off), ref.pitched(dy, ld + 1, off)
        ws, bs = ref.pitched(w[None], 201, off)[0], ref.pitched(b[None], 201, off)[0]
        y, mean, rstd = dg.layer_norm(xs, ws, bs, eps=EPS, return_stats=True)
        ref.check(y, ref.layer_norm(x.double(), w.double(), b.double(), EPS, dtype)[0], "y")
        got = dg.layer_norm_backward(dys, xs, ws, mean, rstd)
        want = ref.layer_norm_backward(dy.double(), x.double(), w.double(), mean.double(),
                                       rstd.double(), None, dtype)
        for g, w_, what in zip(got, want, ("dx", "dweight", "dbias")):
            ref.check(g, w_, f"{what} pitch {ld} offset {off}")
    one, zero = torch.ones_like(w).double(), torch.zeros_like(b).double()
    ref.check(dg.layer_norm(x), ref.layer_norm(x.double(), one, zero, EPS, dtype)[0], "plain")
    ref.check(dg.layer_norm(x, w), ref.layer_norm(x.double(), w.double(), zero, EPS, dtype)[0], "w")


def test_many_leading_dimensions_out_and_empty_input():
    n, x, w, b = _inputs(24, 96, torch.bfloat16, 9)
    y, mean, rstd = dg.layer_norm(x.view(2, 3, 4, 96), w, b, return_stats=True)
    assert y.shape == (2, 3, 4, 96) and mean.shape == rstd.shape == (2, 3, 4)
    assert torch.equal(y.view(24, 96), dg.layer_norm(x, w, b))
    dx, _, _ = dg.layer_norm_backward(y, x.view(2, 3, 4, 96), w, mean, rstd)
    assert dx.shape == (2, 3, 4, 96)
    buf = torch.full((24, 100), 7.0, dtype=torch.bfloat16, device="cuda")
    dg.layer_norm(x, w, b, out=buf[:, 1:97])
    assert torch.equal(buf[:, 1:97], y.view(24, 96))
    assert (buf[:, :1] == 7).all() and (buf[:, 97:] == 7).all()
    e = x[:0]
    ye, me, re = dg.layer_norm(e, w, b, return_stats=True)
    assert ye.shape == (0, 96)
    dxe, dwe, dbe = dg.layer_norm_backward(e, e, w, me, re)  # sums over nothing
    assert dxe.shape == (0, 96) and not dwe.any() and not dbe.any()


def test_constant_rows_and_special_values():
    """A constant row has variance 0: y = bias exactly.  An infinity or NaN stays in its row."""
    w = torch.full((640,), 2.0, device="cuda")
    b = torch.arange(640.0, device="cuda")
    x = torch.full((4, 640), 3.0, device="cuda")
    x[1, 5] = float("inf")
    x[2, 639] = float("nan")
    y = dg.layer_norm(x, w, b)
    assert torch.equal(y[0], b) and torch.equal(y[3], b)
    assert torch.isnan(y[1]).any() and torch.isnan(y[2]).all()


def test_a_row_offset_past_32_bits():
    """Rows that lie more than 2^32 elements into their buffer."""
    cols, ld = 64, 1 << 28
    buf = torch.empty(20 * ld + cols, dtype=torch.float16, device="cuda")
    x = buf.as_strided((21, cols), (ld, 1))
    _, small, w, b = _inputs(21, cols, torch.float16, 3)
    x.copy_(small)
    y, mean, rstd = dg.layer_norm(x, w, b, return_stats=True)
    assert torch.equal(y, dg.layer_norm(small, w, b))
    assert torch.equal(dg.layer_norm_backward(y, x, w, mean, rstd)[0],
                       dg.layer_norm_backward(y, small, w, mean, rstd)[0])


def test_gradient_against_differences():
    """<dx, v> against central differences of the 64-bit forward form."""
    n, x, w, b = _inputs(6, 300, torch.float32, 12)
    c, v = n((6, 300), torch.float32), n((6, 300), torch.float32).double()
    _, mean, rstd = dg.layer_norm(x, w, b, return_stats=True)
    dx, dw, db = dg.layer_norm_backward(c, x, w, mean, rstd)
    f = lambda t: (c.double() * ref.layer_norm(t, w.double(), b.double(), EPS, torch.float32)[0][0]).sum()  # noqa: E731
    h = 1e-4
    want = (f(x.double() + h * v) - f(x.double() - h * v)) / (2 * h)
    # differences: h^2 f''' / 6 ~ 1e-8; fp32 gradient: 1e-5 of sum |dx v|
    assert abs((dx.double() * v).sum() - want) <= 1e-5 * (dx.double() * v).abs().sum() + 1e-6


def test_other_stream():
    n, x, w, b = _inputs(50, 512, torch.bfloat16, 1)
    want = dg.layer_norm(x, w, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        got = dg.layer_norm(x, w, b, stream=stream)
        s.synchronize()
        assert torch.equal(got, want)
    gu.check_watchdog()
