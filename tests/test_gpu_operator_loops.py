"""The persistent kernels of the operators over many rows and tiles, as calls of
training size run them: rings that are refilled several times over, CTA pairs that
take several tiles each, grids that go round their jobs.  Against the 64-bit forms."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import ops_reference as ref

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    torch.cuda.empty_cache()


def _d(t):
    return None if t is None else t.double()


# every width of a row's group of threads (32 to 512), 13 to 26 rows per group and at
# most 8 stages, rows on any alignment
@pytest.mark.parametrize("rows, cols", [(40000, 300), (40003, 301), (16384, 1024), (16385, 1013),
                                        (10000, 2048), (5000, 4096), (5001, 4099), (4000, 8192),
                                        (4001, 8189), (2000, 8200), (2001, 8201), (2001, 16384)])
@pytest.mark.parametrize("dtype", [BF, HF, F32], ids=str)
@pytest.mark.parametrize("skip", [False, True])
def test_layer_norm_backward(rows, cols, dtype, skip):
    n = ref.make(rows + cols)
    x, w, dy = n((rows, cols), dtype, 1.5, 0.25), n((cols,), dtype, 0.2, 1.0), n((rows, cols), dtype, 0.1)
    dr = n((rows, cols), dtype, 0.1) if skip else None
    _, mean, rstd = dg.layer_norm(x, w, None, return_stats=True)
    got = dg.layer_norm_backward(dy, x, w, mean, rstd, dresidual=dr)
    want = ref.layer_norm_backward(_d(dy), _d(x), _d(w), _d(mean), _d(rstd), _d(dr), dtype)
    for g, w_, what in zip(got, want, ("dx", "dweight", "dbias")):
        ref.check(g, w_, f"{what} {rows}x{cols} {dtype}")
    gu.check_watchdog()


# over three tiles for each of 76 pairs in every product, aligned and not
SIZES = [(4100, 4104, 4112), (4099, 4101, 4097)]


@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("M, N, K", SIZES + [(4096, 4096, 136)])
def test_linear(M, N, K, trans_w, monkeypatch):
    monkeypatch.setenv("DGEMM_FUSED_PAIR", "1")
    dtype = HF if trans_w else BF
    n = ref.make(M + N)
    x, w, b, r = n((M, K), dtype), n((K, N), dtype, K ** -0.5), n((N,), dtype, 0.5), n((M, N), dtype)
    ws = w.t().contiguous() if trans_w else w
    d, z = dg.linear(x, ws, b, "gelu", r, trans_w=trans_w, return_preact=True)
    want = ref.linear(_d(x), _d(w), _d(b), "gelu", _d(r), dtype)
    ref.check(d, want[0], "d")
    ref.check(z, want[1], "z")
    del want
    dd = n((M, N), dtype, 0.2)
    got = dg.linear_backward(dd, x, ws, "gelu", z, trans_w=trans_w)
    want = ref.linear_backward(_d(dd), _d(x), _d(w), "gelu", _d(z), dtype)
    for g, w_, what in zip((got[0], got[1].t() if trans_w else got[1], got[2]), want, ("dx", "dw", "db")):
        ref.check(g, w_, what)
    gu.check_watchdog()


@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("M, D, F", SIZES)
def test_gated(M, D, F, trans_w, monkeypatch):
    monkeypatch.setenv("DGEMM_FUSED_PAIR", "1")
    dtype = BF if trans_w else HF
    n = ref.make(M + D)
    x, r, dy = n((M, D), dtype), n((M, D), dtype), n((M, D), dtype, 0.2)
    ws = [n((D, F), dtype, D ** -0.5), n((D, F), dtype, D ** -0.5), n((F, D), dtype, F ** -0.5)]
    wt = [w.t().contiguous() if trans_w else w for w in ws]
    y, g, u = dg.gated_ffn(x, *wt, "silu", r, trans_w=trans_w, return_saved=True)
    want = ref.gated(_d(x), *map(_d, ws), "silu", _d(r), dtype)
    for got, w_, what in zip((y, g, u), want, "ygu"):
        ref.check(got, w_, what)
    del want
    got = dg.gated_ffn_backward(dy, x, *wt, g, u, "silu", trans_w=trans_w)
    want = ref.gated_backward(_d(dy), _d(x), *map(_d, ws), _d(g), _d(u), "silu", dtype)
    for i, (v, w_, what) in enumerate(zip(got, want, ("dx", "dwg", "dwu", "dwd"))):
        ref.check(v.t() if trans_w and i else v, w_, what)
    gu.check_watchdog()


@pytest.mark.parametrize("cols", [296, 301])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_many_rows(cols, act):
    """dz with its column sums over several rounds of rows per warp; with odd columns
    operands are re-pitched by a grid that goes round."""
    M, K = 60000, 63
    n = ref.make(cols)
    x, w, dd, z = n((M, K), BF), n((K, cols), BF, 0.1), n((M, cols), BF, 0.2), n((M, cols), BF)
    got = dg.linear_backward(dd, x, w, act, z)
    want = ref.linear_backward(_d(dd), _d(x), _d(w), act, _d(z), BF)
    for g, w_, what in zip(got, want, ("dx", "dw", "db")):
        ref.check(g, w_, what)
    gu.check_watchdog()
