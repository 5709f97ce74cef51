"""Every kernel and cut a fused product can be given (forced by DGEMM_FUSED_*)
on shapes of partial tiles, against the 64-bit reference."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import ops_reference as ref

pytestmark = pytest.mark.gpu
PLANS = [dict(PAIR=1)] + [dict(PAIR=0, NT=nt, KD=kd, SPLITS=s)
                          for nt, kd, s in ((16, 1, 1), (16, 2, 8), (32, 2, 3), (48, 2, 2), (64, 1, 4),
                                            (64, 2, 6), (96, 1, 2), (128, 1, 8), (192, 1, 2),
                                            (208, 1, 1), (256, 1, 4))]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def _force(monkeypatch, plan):
    for k, v in plan.items():
        monkeypatch.setenv("DGEMM_FUSED_" + k, str(v))


def _d(t):
    return None if t is None else t.double()


@pytest.mark.parametrize("plan", PLANS, ids=str)
@pytest.mark.parametrize("M, N, K", [(1, 136, 200), (130, 264, 1000), (300, 77, 333), (520, 1040, 64)])
@pytest.mark.parametrize("trans_w", [False, True])
def test_linear(M, N, K, trans_w, plan, monkeypatch):
    _force(monkeypatch, plan)
    n = ref.make(M + N)
    dtype = torch.bfloat16 if K % 2 else torch.float16
    x, w = n((M, K), dtype), n((K, N), dtype, K ** -0.5)
    b, r, dd = n((N,), dtype), n((M, N), dtype), n((M, N), dtype, 0.2)
    ws = w.t().contiguous() if trans_w else w
    d, z = dg.linear(x, ws, b, "silu", r, trans_w=trans_w, return_preact=True)
    want = ref.linear(_d(x), _d(w), _d(b), "silu", _d(r), dtype)
    ref.check(d, want[0], "d")
    ref.check(z, want[1], "z")
    got = dg.linear_backward(dd, x, ws, "silu", z, trans_w=trans_w)
    want = ref.linear_backward(_d(dd), _d(x), _d(w), "silu", _d(z), dtype)
    for g, w_, what in zip((got[0], got[1].t() if trans_w else got[1], got[2]), want, ("dx", "dw", "db")):
        ref.check(g, w_, what)
    gu.check_watchdog()


@pytest.mark.parametrize("plan", PLANS, ids=str)
@pytest.mark.parametrize("M, D, F", [(1, 200, 136), (130, 264, 200), (300, 77, 333), (520, 64, 520)])
@pytest.mark.parametrize("trans_w", [False, True])
def test_gated(M, D, F, trans_w, plan, monkeypatch):
    _force(monkeypatch, plan)
    n = ref.make(M + D)
    dtype = torch.bfloat16 if D % 2 else torch.float16
    x, r, dy = n((M, D), dtype), n((M, D), dtype), n((M, D), dtype, 0.2)
    ws = [n((D, F), dtype, D ** -0.5), n((D, F), dtype, D ** -0.5), n((F, D), dtype, F ** -0.5)]
    wt = [w.t().contiguous() if trans_w else w for w in ws]
    y, g, u = dg.gated_ffn(x, *wt, "gelu_tanh", r, trans_w=trans_w, return_saved=True)
    want = ref.gated(_d(x), *map(_d, ws), "gelu_tanh", _d(r), dtype)
    for got, w_, what in zip((y, g, u), want, "ygu"):
        ref.check(got, w_, what)
    got = dg.gated_ffn_backward(dy, x, *wt, g, u, "gelu_tanh", trans_w=trans_w)
    want = ref.gated_backward(_d(dy), _d(x), *map(_d, ws), _d(g), _d(u), "gelu_tanh", dtype)
    for i, (v, w_, what) in enumerate(zip(got, want, ("dx", "dwg", "dwu", "dwd"))):
        ref.check(v.t() if trans_w and i else v, w_, what)
    gu.check_watchdog()


@pytest.mark.parametrize("batch", [0, 1])
@pytest.mark.parametrize("plan", [{}] + PLANS[1::3], ids=str)
@pytest.mark.parametrize("M, D, F", [(1, 200, 136), (97, 130, 264), (300, 77, 333)])
def test_gradients_together_and_apart(M, D, F, plan, batch, monkeypatch):
    """The independent products of a backward pass as one launch, or one each."""
    _force(monkeypatch, dict(plan, BATCH=batch))
    n = ref.make(M + D)
    dtype = torch.float16
    x, dy, g, u = n((M, D), dtype), n((M, D), dtype, 0.2), n((M, F), dtype), n((M, F), dtype)
    ws = [n((D, F), dtype, D ** -0.5), n((D, F), dtype, D ** -0.5), n((F, D), dtype, F ** -0.5)]
    got = dg.gated_ffn_backward(dy, x, *ws, g, u, "silu")
    want = ref.gated_backward(_d(dy), _d(x), *map(_d, ws), _d(g), _d(u), "silu", dtype)
    for v, w_, what in zip(got, want, ("dx", "dwg", "dwu", "dwd")):
        ref.check(v, w_, what)
    n0 = dg.dgemm_kernel_launches()
    got = dg.linear_backward(g, x, ws[0], "none", with_bias=False)
    launched = dg.dgemm_kernel_launches() - n0
    want = ref.linear_backward(_d(g), _d(x), _d(ws[0]), "none", None, dtype)
    for v, w_, what in zip(got, want, ("dx", "dw")):
        ref.check(v, w_, what)
    if D % 8 == 0 and F % 8 == 0:  # nothing to stage
        assert launched == (1 if batch else 2)
    gu.check_watchdog()
