"""The gated feed-forward block on the GPU, forward and backward, against the
64-bit reference within bounds derived in ops_reference.py."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import ops_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16]
GATES = ("none", "relu", "gelu", "gelu_tanh", "silu")
# (M, D, F): one token, a few, around tile edges, odd everywhere, large enough
# for many tiles
SHAPES = [(1, 64, 128), (1, 1024, 1000), (2, 1, 8), (3, 17, 1), (16, 136, 520), (33, 129, 65),
          (64, 512, 2048), (100, 257, 1000), (129, 300, 72), (256, 128, 64), (300, 997, 1013),
          (1000, 520, 1032), (2100, 264, 700)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def _d(t):
    return None if t is None else t.double()


def _block(M, D, F, dtype, seed):
    n = ref.make(seed)
    return (n, n((M, D), dtype), n((D, F), dtype, max(D, 1) ** -0.5),
            n((D, F), dtype, max(D, 1) ** -0.5), n((F, D), dtype, max(F, 1) ** -0.5))


def _t(ws, trans_w):
    return [w.t().contiguous() if trans_w else w for w in ws]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("M, D, F", SHAPES)
def test_forward(M, D, F, trans_w, dtype):
    act = GATES[(M + D + F) % 5]
    n, x, *ws = _block(M, D, F, dtype, M + D + F)
    r = n((M, D), dtype)
    y, g, u = dg.gated_ffn(x, *_t(ws, trans_w), act, r, trans_w=trans_w, return_saved=True)
    want = ref.gated(_d(x), *map(_d, ws), act, _d(r), dtype)
    for got, w_, what in zip((y, g, u), want, "ygu"):
        ref.check(got, w_, f"{what} {act}")
    assert torch.equal(dg.gated_ffn(x, *_t(ws, trans_w), act, r, trans_w=trans_w), y)
    ref.check(dg.gated_ffn(x, *_t(ws, trans_w), act, trans_w=trans_w),
              ref.gated(_d(x), *map(_d, ws), act, None, dtype)[0], "no residual")
    gu.check_watchdog()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("trans_w", [False, True])
@pytest.mark.parametrize("M, D, F", SHAPES)
def test_backward(M, D, F, trans_w, dtype):
    act = GATES[(M + 2 * D + F) % 5]
    n, x, *ws = _block(M, D, F, dtype, M + D + F)
    dy, g, u = n((M, D), dtype, 0.2), n((M, F), dtype), n((M, F), dtype)
    got = dg.gated_ffn_backward(dy, x, *_t(ws, trans_w), g, u, act, trans_w=trans_w)
    want = ref.gated_backward(_d(dy), _d(x), *map(_d, ws), _d(g), _d(u), act, dtype)
    for i, (v, w_, what) in enumerate(zip(got, want, ("dx", "dwg", "dwu", "dwd"))):
        ref.check(v.t() if trans_w and i else v, w_, f"{what} {act}")
    again = dg.gated_ffn_backward(dy, x, *_t(ws, trans_w), g, u, act, trans_w=trans_w)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    gu.check_watchdog()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M", [4, 320])
@pytest.mark.parametrize("act", GATES)
def test_every_activation(act, M, dtype):
    n, x, *ws = _block(M, 72, 136, dtype, 11)
    x = x * 3  # out to where the activations saturate
    ref.check(dg.gated_ffn(x, *ws, act), ref.gated(_d(x), *map(_d, ws), act, None, dtype)[0], act)
    dy, g, u = n((M, 72), dtype), n((M, 136), dtype, 3.0), n((M, 136), dtype)
    got = dg.gated_ffn_backward(dy, x, *ws, g, u, act)
    want = ref.gated_backward(_d(dy), _d(x), *map(_d, ws), _d(g), _d(u), act, dtype)
    for v, w_, what in zip(got, want, ("dx", "dwg", "dwu", "dwd")):
        ref.check(v, w_, f"{what} {act}")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("M, D, F", [(3, 72, 80), (70, 130, 200), (520, 264, 392)])
@pytest.mark.parametrize("pad, offset", [(0, 8), (8, 0), (3, 1)])
def test_strides_and_alignment(M, D, F, pad, offset, dtype):
    n, x, *ws = _block(M, D, F, dtype, 5)
    r, dy, g, u = n((M, D), dtype), n((M, D), dtype), n((M, F), dtype), n((M, F), dtype)
    p = lambda t: ref.pitched(t, t.shape[1] + pad, offset)  # noqa: E731
    out = torch.full((M, D + pad), 7.0, dtype=dtype, device="cuda")[:, :D]
    y = dg.gated_ffn(p(x), *map(p, ws), "silu", p(r), out=out)
    ref.check(y, ref.gated(_d(x), *map(_d, ws), "silu", _d(r), dtype)[0], "y")
    got = dg.gated_ffn_backward(p(dy), p(x), *map(p, ws), p(g), p(u), "silu")
    want = ref.gated_backward(_d(dy), _d(x), *map(_d, ws), _d(g), _d(u), "silu", dtype)
    for v, w_, what in zip(got, want, ("dx", "dwg", "dwu", "dwd")):
        ref.check(v, w_, what)


@pytest.mark.parametrize("M", [1, 400])
def test_residual_in_place(M):
    n, x, *ws = _block(M, 136, 264, torch.bfloat16, 3)
    r = n((M, 136), torch.bfloat16)
    want = dg.gated_ffn(x, *ws, residual=r)
    assert dg.gated_ffn(x, *ws, residual=r, out=r) is r and torch.equal(r, want)


def test_empty_shapes():
    bf = torch.bfloat16
    _, x, *ws = _block(0, 16, 24, bf, 1)
    assert dg.gated_ffn(x, *ws).shape == (0, 16)
    f0 = x.new_zeros((0, 24))
    dx, *dws = dg.gated_ffn_backward(x, x, *ws, f0, f0)
    assert dx.shape == (0, 16) and not any(w.any() for w in dws)
    n, x, *ws = _block(5, 16, 0, bf, 1)
    r = n((5, 16), bf)
    assert torch.equal(dg.gated_ffn(x, *ws, residual=r), r)
    f0 = x.new_zeros((5, 0))
    dx, *dws = dg.gated_ffn_backward(x, x, *ws, f0, f0)
    assert not dx.any() and all(w.numel() == 0 for w in dws)
    _, x, *ws = _block(5, 0, 24, bf, 1)
    y, g, u = dg.gated_ffn(x, *ws, return_saved=True)
    assert y.shape == (5, 0) and not g.any() and not u.any()


def test_gradients_against_differences():
    """<grad, v> against central differences of the 64-bit forward form."""
    n, x, *ws = _block(20, 32, 48, torch.float16, 4)
    c = n((20, 32), torch.float16)
    args = [_d(x), *map(_d, ws)]
    _, (g, _), (u, _) = ref.gated(*args, "silu", None, torch.float16)
    got = dg.gated_ffn_backward(c, x, *ws, g.half(), u.half(), "silu")
    f = lambda *t: (_d(c) * ref.gated(*t, "silu", None, torch.float16)[0][0]).sum()  # noqa: E731
    h = 1e-5
    for i in range(4):
        v = n(args[i].shape, torch.float32).double()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * v, args[i] - h * v
        want = (f(*up) - f(*down)) / (2 * h)
        # g, u, the workspaces and the gradient round by 2^-11 each: below 2^-9 of sum |grad v|
        assert abs((_d(got[i]) * v).sum() - want) <= 2.0 ** -9 * (_d(got[i]) * v).abs().sum()


def test_streams_do_not_mix():
    """Calls on two streams at once give what they give alone."""
    n, x, *ws = _block(200, 256, 512, torch.bfloat16, 3)
    n2, x2, *ws2 = _block(200, 256, 512, torch.bfloat16, 4)
    want, want2 = dg.gated_ffn(x, *ws), dg.gated_ffn(x2, *ws2)
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a, b = dg.gated_ffn(x, *ws, stream=s), dg.gated_ffn(x2, *ws2, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want2)
