"""The products in 8-bit integers on the GPU against the 64-bit reference
within the bounds of int8_reference.py."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import int8_reference as ref8
import ops_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]
ALL = DTYPES + [torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    gu.check_watchdog()


def _d(t):
    return None if t is None else t.double()


def _ints(n, rows, cols, seed=0):
    """A weight in 8 bits with the float32 scales of its rows."""
    gen = torch.Generator().manual_seed(seed + rows + 3 * cols)
    w = torch.randint(-127, 128, (rows, cols), generator=gen, dtype=torch.int8).cuda()
    return w, n((rows,), torch.float32, 0.1, 1.0).abs() * (0.01 * max(cols, 1) ** -0.5)


# ------------------------------------------------------------------ quantize_int8
@pytest.mark.parametrize("dtype", ALL, ids=str)
@pytest.mark.parametrize("rows, cols", [(1, 1), (3, 7), (5, 64), (2, 997), (300, 1024), (4, 4096), (3, 4100),
                                        (2, 8200), (2, 40001)])
def test_rows_in_8_bits(rows, cols, dtype):
    x = ref.make(rows + cols)((rows, cols), dtype)
    q, s = dg.quantize_int8(x)
    want, scale = ref8.quantize(x)
    assert q.dtype == torch.int8 and s.dtype == torch.float32 and s.shape == (rows,)
    # 53 bits are enough for a second rounding to be that of the quotient (torch's own
    # fp32 division by a number is a product with its reciprocal on the GPU)
    assert torch.equal(s, scale.float())
    if dtype != torch.float32:
        assert torch.equal(q.double(), want)
    else:  # the quotient in fp32: 2^-24 of 127 from the exact one, twice
        t = 127.0 * x.double() / x.double().abs().amax(1, keepdim=True)
        assert bool(((q.double() - t).abs() <= 0.5 + 2.0 ** -16).all())


@pytest.mark.parametrize("dtype", ALL, ids=str)
@pytest.mark.parametrize("rows, cols", [(1, 1), (7, 3), (64, 64), (997, 130), (1000, 1013), (4096, 96)])
def test_columns_as_rows(rows, cols, dtype):
    x = ref.make(rows + cols)((rows, cols), dtype)
    q, s = dg.quantize_int8(x, transpose=True)
    qt, st = dg.quantize_int8(x.t().contiguous())
    assert torch.equal(q, qt) and torch.equal(s, st)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_halves_go_to_the_even_integer(dtype):
    # 127 x / top is k + 1/2 exactly for x = (2 k + 1) top / 254: top 127, x a multiple of 1/2
    k = torch.arange(-127, 127, dtype=torch.float64)
    x = torch.cat([k + 0.5, torch.tensor([127.0], dtype=torch.float64)]).to(dtype).cuda()[None]
    got = dg.quantize_int8(x)[0][0, :-1].double().cpu()
    assert torch.equal(got, torch.round(x[0, :-1].double().cpu()))


def test_every_bfloat16_against_every_top_of_a_binade():
    """All 2^15 sizes from 0 to the largest of a row, for tops across the exponents."""
    bits = torch.arange(0, 0x7f80, dtype=torch.int32)
    every = bits.to(torch.int16).view(torch.bfloat16).cuda()
    for top in (0x0001, 0x0040, 0x0080, 0x00ff, 0x3f80, 0x3fab, 0x40ff, 0x7e80, 0x7f00, 0x7f7f):
        x = torch.cat([every[: top + 1], -every[: top + 1]])[None]
        q, s = dg.quantize_int8(x)
        assert torch.equal(q.double(), ref8.quantize(x)[0]), hex(top)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype", ALL, ids=str)
def test_rows_without_a_scale(dtype, transpose):
    x = ref.make(3)((6, 200), dtype)
    x[1], x[2, 5], x[3, 7], x[4, 9] = 0, float("inf"), float("nan"), float("-inf")
    q, s = dg.quantize_int8(x.t().contiguous(), transpose=True) if transpose else dg.quantize_int8(x)
    assert bool((q[1:5] == 0).all()) and s[1] == 0 and s[2] == float("inf") and s[4] == float("inf")
    assert torch.isnan(s[3])
    assert torch.equal(q[::5].double(), ref8.quantize(x[::5])[0]) or dtype == torch.float32


def test_quantize_shapes_strides_and_nothing():
    n = ref.make(9)
    x = n((2, 3, 40), torch.bfloat16)
    q, s = dg.quantize_int8(x)
    assert q.shape == x.shape and s.shape == (2, 3)
    assert torch.equal(q.view(6, 40).double(), ref8.quantize(x.view(6, 40))[0])
    y = ref.pitched(n((33, 51), torch.float16), 59, 3)
    assert torch.equal(dg.quantize_int8(y)[0].double(), ref8.quantize(y)[0])
    assert torch.equal(dg.quantize_int8(y, transpose=True)[0].double(), ref8.quantize(y.t())[0])
    q, s = dg.quantize_int8(x[:0].view(0, 40))
    assert q.shape == (0, 40) and s.shape == (0,)
    q, s = dg.quantize_int8(torch.empty((3, 0), device="cuda"))
    assert q.shape == (3, 0) and torch.equal(s, torch.zeros(3, device="cuda"))
    q, s = dg.quantize_int8(torch.empty((0, 3), device="cuda"), transpose=True)
    assert q.shape == (3, 0) and torch.equal(s, torch.zeros(3, device="cuda"))


# -------------------------------------------------------------------- linear_int8
SHAPES = [(1, 64, 64), (1, 1000, 4096), (2, 8, 1), (3, 1, 17), (16, 136, 520), (17, 129, 65),
          (64, 512, 2048), (100, 257, 1000), (128, 128, 128), (129, 300, 72), (255, 96, 333),
          (257, 512, 64), (1000, 1013, 997), (700, 2048, 256), (2100, 1032, 130), (1, 4096, 14336)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("M, N, K", SHAPES)
def test_linear(M, N, K, given, dtype):
    n = ref.make(M + N + K)
    x, (w, ws) = n((M, K), dtype), _ints(n, N, K)
    act = ref.ACTS[(M + N + K) % 5]
    b = n((N,), dtype, 0.5) if (M + K) % 3 else None
    r = n((M, N), dtype) if (N + K) % 2 else None
    q, s = ref8.quantize(x)
    want = ref8.linear(q, s, _d(w), _d(ws), _d(b), act, _d(r), dtype)
    if given:
        xq, xs = dg.quantize_int8(x)
        got = dg.linear_int8(xq, w, ws, b, act, r, x_scale=xs, dtype=dtype)
    else:
        got = dg.linear_int8(x, w, ws, b, act, r)
    ref.check(got, want, f"{act} bias={b is not None} residual={r is not None}")
    again = dg.linear_int8(x, w, ws, b, act, r)
    assert torch.equal(again, got)


@pytest.mark.parametrize("M, N, K", [(40, 264, 700), (300, 530, 390)])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_linear_rows_of_any_pitch_and_alignment(M, N, K, dtype):
    n = ref.make(M)
    x, (w, ws) = n((M, K), dtype), _ints(n, N, K)
    r, b = n((M, N), dtype), n((N,), dtype)
    want = dg.linear_int8(x, w, ws, b, "silu", r)
    for off, pad in ((1, 3), (2, 6), (8, 8), (3, 13)):
        wide = torch.zeros(off + N * (K + pad), dtype=torch.int8, device="cuda")
        w2 = wide.as_strided((N, K), (K + pad, 1), off)
        w2.copy_(w)
        x2, r2 = ref.pitched(x, K + pad, off), ref.pitched(r, N + pad, off)
        out = ref.pitched(r, N + pad, off)
        got = dg.linear_int8(x2, w2, ws, b, "silu", r2, out=out)
        assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
        inner = out.as_strided((M - 1, pad), (N + pad, 1), off + N)
        assert bool(torch.isnan(inner).all()), "written between the rows"
        xq, xs = dg.quantize_int8(x)
        q2 = torch.zeros(off + M * (K + pad), dtype=torch.int8, device="cuda").as_strided((M, K), (K + pad, 1), off)
        q2.copy_(xq)
        assert torch.equal(dg.linear_int8(q2, w2, ws, b, "silu", r2, x_scale=xs, dtype=dtype), want)
    dg.linear_int8(x, w, ws, b, "silu", r, out=r)  # the residual itself
    assert torch.equal(r, want)


def test_linear_leading_dimensions_and_empty():
    n = ref.make(4)
    x, (w, ws) = n((2, 5, 96), torch.bfloat16), _ints(n, 40, 96)
    y = dg.linear_int8(x, w, ws)
    assert y.shape == (2, 5, 40) and torch.equal(y.view(10, 40), dg.linear_int8(x.view(10, 96), w, ws))
    v = dg.linear_int8(x[0, 0], w, ws)
    assert v.shape == (40,) and torch.equal(v, dg.linear_int8(x[0, :1], w, ws)[0])
    assert dg.linear_int8(x[:0], w, ws).shape == (0, 5, 40)
    assert dg.linear_int8(x, w[:0], ws[:0]).shape == (2, 5, 0)
    b, r = n((40,), torch.bfloat16), n((3, 40), torch.bfloat16)
    none = dg.linear_int8(x[0, :3, :0], w[:, :0], ws, b, "relu", r)  # an empty sum is zero
    assert torch.equal(none, (b.float().clamp(min=0) + r.float()).bfloat16())


@pytest.mark.parametrize("M", [1, 200, 600])
def test_linear_largest_integers_and_extreme_rows(M):
    """Sums past 2^24, the lowest byte, tokens at the ends of bfloat16's range, rows without a scale."""
    K, N = 4096, 320
    w = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    w[1::4], w[2::4] = -128, -127
    w[3::4, ::2] = -127
    ws = torch.full((N,), 2.0 ** -20, device="cuda")
    x = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    q, s = ref8.quantize(x)
    ref.check(dg.linear_int8(x, w, ws), ref8.linear(q, s, _d(w), _d(ws), None, "none", None, torch.bfloat16), "127")
    x = ref.make(2)((M, K), torch.bfloat16)
    x[0] *= 2.0 ** 126 / x[0].abs().max().float()
    if M > 1:
        x[1] *= 2.0 ** -126 / x[1].abs().max().float()
        x[2], x[3, 70], x[4, 3] = 0, float("nan"), float("-inf")
    got = dg.linear_int8(x, w, ws)
    q, s = ref8.quantize(x)
    value, bound = ref8.linear(q, s, _d(w), _d(ws), None, "none", None, torch.bfloat16)
    # the smallest row's scale is a subnormal float: half its last place, times the sum
    bound[1:2] += 2.0 ** -150 * (q.abs() @ _d(w).abs().T * _d(ws))[1:2]
    fine = [i for i in range(M) if i not in (3, 4)]
    ref.check(got[fine], (value[fine], bound[fine]), "extreme rows")
    if M > 1:
        assert bool((got[2] == 0).all()) and bool(torch.isnan(got[3:5]).all())


# ----------------------------------------------------------------- gated_ffn_int8
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M, D, F", [(1, 64, 128), (1, 4096, 1408), (3, 40, 24), (17, 130, 257), (64, 1024, 4096),
                                     (200, 264, 520), (130, 997, 1013), (700, 256, 1032)])
def test_gated(M, D, F, dtype):
    n = ref.make(M + D + F)
    x = n((M, D), dtype)
    act = ref.ACTS[1 + (M + D) % 4]
    (wg, sg), (wu, su), (wd, sd) = _ints(n, F, D), _ints(n, F, D, 1), _ints(n, D, F, 2)
    r = n((M, D), dtype) if F % 2 == 0 else None
    got = dg.gated_ffn_int8(x, wg, sg, wu, su, wd, sd, act, r)
    ref.check(got, ref8.gated(_d(x), _d(wg), _d(sg), _d(wu), _d(su), _d(wd), _d(sd), act, _d(r), dtype), act)
    assert torch.equal(dg.gated_ffn_int8(x, wg, sg, wu, su, wd, sd, act, r), got)
    if r is not None:
        assert dg.gated_ffn_int8(x, wg, sg, wu, su, wd, sd, act, r, out=r) is not None and torch.equal(r, got)


def test_gated_empty_and_zero_rows():
    n = ref.make(8)
    x = n((5, 48), torch.float16)
    (wg, sg), (wu, su), (wd, sd) = _ints(n, 32, 48), _ints(n, 32, 48, 1), _ints(n, 48, 32, 2)
    assert dg.gated_ffn_int8(x[:0], wg, sg, wu, su, wd, sd).shape == (0, 48)
    r = n((5, 48), torch.float16)
    nothing = dg.gated_ffn_int8(x, wg[:0], sg[:0], wu[:0], su[:0], wd[:, :0], sd, residual=r)
    assert torch.equal(nothing, r)  # no hidden units
    x[2] = 0
    y = dg.gated_ffn_int8(x, wg, sg, wu, su, wd, sd, residual=r)
    assert torch.equal(y[2], r[2])


def test_block_quantised_from_its_weights():
    """The use: a 16-bit block's weights put into 8 bits once, then served; against
    the block in 64 bits on the values that the integers stand for."""
    n = ref.make(11)
    D, F, M = 512, 1408, 40
    x = n((M, D), torch.bfloat16)
    wg, wu, wd = (n(s, torch.bfloat16, s[0] ** -0.5) for s in ((D, F), (D, F), (F, D)))
    q = [dg.quantize_int8(w, transpose=True) for w in (wg, wu, wd)]
    h, mean, rstd = dg.layer_norm(x, return_stats=True)
    y = dg.gated_ffn_int8(h, *q[0], *q[1], *q[2], residual=x)
    ref.check(y, ref8.gated(_d(h), *(t.double() for p in q for t in p), "silu", _d(x), torch.bfloat16), "y")
    full = dg.gated_ffn(h, wg, wu, wd, residual=x)
    off = (y.float() - full.float()).norm() / (full.float() - x.float()).norm()
    assert off < 0.03, float(off)  # 8 bits: 1/254 of a row's largest, some 3.5 sizes of the others, three times


def test_two_streams_and_a_graph():
    n = ref.make(12)
    x, (w, ws) = n((48, 512), torch.bfloat16), _ints(n, 300, 512)
    want = dg.linear_int8(x, w, ws)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[dg.linear_int8(x, w, ws, stream=s) for _ in range(20)] for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for os in outs for o in os)
    graphs, results = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(dg.linear_int8(x, w, ws, activation="none"))
        graphs.append(g)
    x.copy_(n((48, 512), torch.bfloat16))
    torch.cuda.synchronize()
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    want = dg.linear_int8(x, w, ws)
    assert all(torch.equal(r, want) for r in results)


@pytest.mark.parametrize("plan", [dict(SPLITS=1, NT=16), dict(SPLITS=1, NT=128), dict(SPLITS=3, NT=48),
                                  dict(SPLITS=8, NT=64)], ids=str)
@pytest.mark.parametrize("M, N, K", [(70, 300, 1500), (130, 140, 384)])
def test_every_cut_gives_the_same(M, N, K, plan, monkeypatch):
    """Sums within 2^24 are exact, so any split of K gives the same bits."""
    n = ref.make(M)
    x, (w, ws) = n((M, K), torch.float16), _ints(n, N, K)
    (wu, su), (wd, sd) = _ints(n, N, K, 1), _ints(n, K, N, 2)
    w, wu, wd = (torch.div(t, 16, rounding_mode="trunc") for t in (w, wu, wd))  # 127 * 8 * 1500 < 2^24
    r = n((M, K), torch.float16)
    want = dg.linear_int8(x, w, ws, activation="gelu")
    block = dg.gated_ffn_int8(x, w, ws, wu, su, wd, sd, residual=r)
    monkeypatch.setenv("DGEMM_INT8_PAIR", "0")
    for k, v in plan.items():
        monkeypatch.setenv("DGEMM_INT8_" + k, str(v))
    assert torch.equal(dg.linear_int8(x, w, ws, activation="gelu"), want)
    assert torch.equal(dg.gated_ffn_int8(x, w, ws, wu, su, wd, sd, residual=r), block)


@pytest.mark.parametrize("row", ["0", "1"])
@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("N, K", [(5, 1), (40, 15), (33, 16), (300, 31), (700, 130), (64, 511), (1300, 997), (2500, 1024),
                                  (100, 4096), (90, 4099), (50, 14336), (30, 20001), (9, 32768), (7, 40000)])
def test_few_tokens(M, N, K, row, monkeypatch):
    """Rows of every length that a warp, several warps or none of them hold, on either kernel."""
    monkeypatch.setenv("DGEMM_INT8_ROW", row)
    n = ref.make(M + N + K)
    dtype = DTYPES[(M + K) % 2]
    x, (w, ws) = n((M, K), dtype), _ints(n, N, K)
    b, r = n((N,), dtype, 0.5), n((M, N), dtype)
    q, s = ref8.quantize(x)
    want = ref8.linear(q, s, _d(w), _d(ws), _d(b), "silu", _d(r), dtype)
    got = dg.linear_int8(x, w, ws, b, "silu", r)
    ref.check(got, want, "x")
    xq, xs = dg.quantize_int8(x)
    assert torch.equal(dg.linear_int8(xq, w, ws, b, "silu", r, x_scale=xs, dtype=dtype), got)
    wide = torch.full((N * (K + 5) + 3,), 77, dtype=torch.int8, device="cuda")
    w2 = wide.as_strided((N, K), (K + 5, 1), 3)
    w2.copy_(w)
    assert torch.equal(dg.linear_int8(x, w2, ws, b, "silu", r), got)


@pytest.mark.parametrize("row", ["0", "1"])
@pytest.mark.parametrize("M, D, F", [(1, 64, 96), (2, 1000, 3000), (3, 257, 131), (4, 512, 1408), (1, 2048, 33000)])
def test_few_tokens_through_the_block(M, D, F, row, monkeypatch):
    monkeypatch.setenv("DGEMM_INT8_ROW", row)
    n = ref.make(M + D + F)
    dtype = DTYPES[M % 2]
    x, r = n((M, D), dtype), n((M, D), dtype)
    (wg, sg), (wu, su), (wd, sd) = _ints(n, F, D), _ints(n, F, D, 1), _ints(n, D, F, 2)
    want = ref8.gated(_d(x), _d(wg), _d(sg), _d(wu), _d(su), _d(wd), _d(sd), "gelu", _d(r), dtype)
    ref.check(dg.gated_ffn_int8(x, wg, sg, wu, su, wd, sd, "gelu", r), want, "y")
    x[0] = 0
    y = dg.gated_ffn_int8(x, wg, sg, wu, su, wd, sd, "gelu", r)
    assert torch.equal(y[0], r[0])


def test_few_tokens_rows_without_a_scale():
    n = ref.make(21)
    x, (w, ws) = n((4, 300), torch.bfloat16), _ints(n, 70, 300)
    x[1], x[2, 9], x[3, 1] = 0, float("inf"), float("nan")
    y = dg.linear_int8(x, w, ws)
    assert bool((y[1] == 0).all()) and bool(torch.isnan(y[2:]).all()) and bool(torch.isfinite(y[0]).all())


def test_weights_quantised_just_before_a_single_token():
    """The kernel that writes the weights is the one ahead of the product that reads them."""
    n = ref.make(22)
    x, w = n((1, 2048), torch.bfloat16), n((4096, 2048), torch.bfloat16)
    q, s = dg.quantize_int8(w)
    want = dg.linear_int8(x, q, s)
    for M in (1, 8, 300):
        xs = x.expand(M, -1).contiguous()
        for _ in range(10):
            again, scale = dg.quantize_int8(w)
            assert torch.equal(dg.linear_int8(xs, again, scale)[M - 1:], want)
            again.zero_()


def test_rows_of_quantised_weights_are_aligned():
    n = ref.make(23)
    for x in (n((7, 33), torch.float16), n((2, 3, 50), torch.bfloat16), n((5,), torch.float32), n((4, 32), torch.float32)):
        q, s = dg.quantize_int8(x)
        assert q.shape == x.shape and q.stride(-1) == 1 and q.data_ptr() % 16 == 0
        assert x.dim() == 1 or q.stride(-2) % 16 == 0
        same, again = dg.quantize_int8(x.clone())
        assert torch.equal(q, same) and torch.equal(s, again)
    q, _ = dg.quantize_int8(n((33, 7), torch.float16), transpose=True)
    assert q.shape == (7, 33) and q.stride() == (48, 1)


@pytest.mark.parametrize("M, K, N", [(2048, 4096, 14336), (1000, 1008, 30000), (3, 4096, 14336), (64, 14336, 4096),
                                     (64, 4096, 14336), (200, 4096, 14336), (40, 2001, 20000),
                                     (600, 2001, 20000)])
def test_one_weight_after_the_other(M, K, N):
    """Weights that alternate come from memory, not from L2: nothing is read before it
    has arrived, or after its place was given to the next block."""
    n = ref.make(M + N)
    x = n((M, K), torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(N)
    # |q w| sums to at most 2^24: the integers' sums are exact
    top = min(127, 2 ** 24 // (127 * K))
    ws = [torch.randint(-top, top + 1, (N, K), generator=gen, dtype=torch.int8, device="cuda") for _ in range(4)]
    scale = n((N,), torch.float32, 0.001, 0.002).abs() + 1e-4
    want = [ref8.linear(*ref8.quantize(x), w.double(), scale.double(), None, "none", None, torch.bfloat16) for w in ws]
    for _ in range(4):
        got = [dg.linear_int8(x, w, scale) for w in ws]
        for y, (d, bound) in zip(got, want):
            assert bool(((y.double() - d).abs() <= bound).all())


@pytest.mark.parametrize("M, D, F", [(700, 2048, 8192), (700, 1001, 6007), (30, 1001, 6007)])
def test_one_block_after_the_other(M, D, F):
    n = ref.make(M)
    x = n((M, D), torch.bfloat16)
    blocks = [[t for w in (n((F, D), torch.bfloat16, 0.05), n((F, D), torch.bfloat16, 0.05),
                           n((D, F), torch.bfloat16, 0.05)) for t in (v.contiguous() for v in dg.quantize_int8(w))]
              for _ in range(4)]
    want = [ref8.gated(x, *(_d(t) for t in b), "silu", None, torch.bfloat16) for b in blocks]
    for _ in range(4):
        got = [dg.gated_ffn_int8(x, *b, "silu") for b in blocks]
        for y, (d, bound) in zip(got, want):
            assert bool(((y.double() - d).abs() <= bound).all())


@pytest.mark.parametrize("nt", [32, 64, 96, 128, 160, 192])
@pytest.mark.parametrize("M, N, K", [(70, 300, 1500), (500, 900, 384), (33, 4, 20), (191, 513, 129)])
def test_every_pair_cut_gives_the_same(M, N, K, nt, monkeypatch):
    n = ref.make(M)
    x, (w, ws) = n((M, K), torch.float16), _ints(n, N, K)
    (wu, su), (wd, sd) = _ints(n, N, K, 1), _ints(n, K, N, 2)
    w, wu, wd = (torch.div(t, 16, rounding_mode="trunc") for t in (w, wu, wd))  # 127 * 8 * 1500 < 2^24
    r, b = n((M, K), torch.float16), n((N,), torch.float16)
    monkeypatch.setenv("DGEMM_INT8_ROW", "0")
    monkeypatch.setenv("DGEMM_INT8_PAIR", "0")
    want = dg.linear_int8(x, w, ws, bias=b, activation="silu")
    block = dg.gated_ffn_int8(x, w, ws, wu, su, wd, sd, residual=r)
    monkeypatch.setenv("DGEMM_INT8_PAIR", "1")
    monkeypatch.setenv("DGEMM_INT8_NT", str(nt))
    assert torch.equal(dg.linear_int8(x, w, ws, bias=b, activation="silu"), want)
    assert torch.equal(dg.gated_ffn_int8(x, w, ws, wu, su, wd, sd, residual=r), block)


def test_blocks_on_streams_and_graphs_at_once():
    M, D, F = 96, 512, 1408
    n = ref.make(3)
    xs = [n((M, D), torch.bfloat16) for _ in range(4)]
    weights = [t for s in ((F, D), (F, D), (D, F)) for t in dg.quantize_int8(n(s, torch.bfloat16, 0.05))]
    want = [dg.gated_ffn_int8(x, *weights, residual=x) for x in xs]
    graphs, outs = [], []
    for x in xs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dg.gated_ffn_int8(x, *weights, residual=x))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        late = [dg.gated_ffn_int8(x, *weights, residual=x, stream=s) for x, s in zip(xs[2:], streams[2:])]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs + late, want))
