"""The orthogonalised update on the GPU against the 64-bit formula, within what
newton_reference.py derives."""
import math
import re
import time

import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import newton_reference as nr
import ops_reference as ref

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    gu.check_watchdog()


def _gradient(rows, cols, dtype, seed=0, size=1e-3):
    n = ref.make(seed + rows + cols)
    rank = max(1, min(rows, cols) // 8)
    g = n((rows, rank), torch.float32) @ n((rank, cols), torch.float32, rank ** -0.5)
    return ((g + n((rows, cols), torch.float32, 0.3)) * size).to(dtype)


SHAPES = [(1, 1), (1, 300), (300, 1), (2, 3), (17, 5), (64, 64), (100, 40), (128, 300), (256, 256), (257, 255),
          (512, 1408), (513, 100), (96, 2000), (1013, 997), (700, 2000), (1500, 600)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows, cols", SHAPES)
def test_against_the_formula(rows, cols, dtype):
    x = _gradient(rows, cols, dtype)
    got = dg.orthogonalize(x)
    assert got.dtype == dtype and got.shape == x.shape
    off = nr.check(got, x)
    assert off < 0.005 or min(rows, cols) < 64, off  # a few singular values: chance decides
    assert torch.equal(dg.orthogonalize(x), got)


@pytest.mark.parametrize("rows, cols", [(200, 600), (600, 200), (300, 310)])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7, 10])
def test_steps(steps, rows, cols):
    x = _gradient(rows, cols, torch.bfloat16, steps)
    nr.check(dg.orthogonalize(x, steps=steps), x, steps)


@pytest.mark.parametrize("rows, cols", [(128, 512), (520, 130), (256, 256)])
def test_coefficients_of_each_step(rows, cols):
    # the odd quintic that is steepest at 0 first, then gentler ones, then (15, -10, 3) / 8, which keeps 1 at 1
    c = [(8.2, -22.5, 15.9), (4.1, -2.9, 0.55), (3.9, -2.8, 0.53), (15 / 8, -10 / 8, 3 / 8), (15 / 8, -10 / 8, 3 / 8)]
    x = _gradient(rows, cols, torch.float16, 3)
    nr.check(dg.orthogonalize(x, coefficients=c), x, 5, c)
    nr.check(dg.orthogonalize(x, steps=2, coefficients=c[2:4]), x, 2, c[2:4])
    nr.check(dg.orthogonalize(x, steps=3, coefficients=[0.0, 0.0, 0.0]), x, 3, (0.0, 0.0, 0.0))


@pytest.mark.parametrize("plan", [dict(PAIR=1), dict(PAIR=0, SPLITS=1), dict(PAIR=0, SPLITS=2), dict(PAIR=0, SPLITS=4),
                                  dict(PAIR=0, SPLITS=8)], ids=str)
@pytest.mark.parametrize("rows, cols", [(40, 60), (260, 700), (700, 260), (530, 520), (513, 1030)])
def test_every_kernel_and_cut(rows, cols, plan, monkeypatch):
    for k, v in plan.items():
        monkeypatch.setenv("DGEMM_NEWTON_" + k, str(v))
    for x_type, w_type in ((torch.bfloat16, torch.float32), (torch.float16, torch.float16)):
        x, w = _gradient(rows, cols, x_type, 1), ref.make(2)((rows, cols), w_type, rows ** -0.5)
        got = dg.orthogonalize(x, scale=-0.02, residual=w, residual_scale=0.998)
        nr.check(got, x, scale=-0.02, residual=w, keep=0.998)
        assert torch.equal(dg.orthogonalize(x, scale=-0.02, residual=w, residual_scale=0.998), got)


@pytest.mark.parametrize("x_type", TYPES, ids=str)
@pytest.mark.parametrize("w_type", TYPES, ids=str)
@pytest.mark.parametrize("rows, cols", [(130, 520), (520, 130), (300, 1001)])
def test_update_of_weights(rows, cols, w_type, x_type):
    x, w = _gradient(rows, cols, x_type, 1), ref.make(2)((rows, cols), w_type, rows ** -0.5)
    args = dict(scale=-0.02, residual=w, residual_scale=0.998)
    got = dg.orthogonalize(x, **args)
    assert got.dtype == w_type
    nr.check(got, x, scale=-0.02, residual=w, keep=0.998)
    out = torch.empty_like(w)
    assert dg.orthogonalize(x, **args, out=out) is not None and torch.equal(out, got)
    plain = dg.orthogonalize(x, out=torch.empty_like(w))
    assert plain.dtype == w_type
    nr.check(plain, x)
    dg.orthogonalize(x, scale=-0.02, residual=w, residual_scale=0.998, out=w)  # in place
    assert torch.equal(w, got)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows, cols", [(70, 333), (333, 70), (260, 264)])
def test_rows_of_any_pitch_and_alignment(rows, cols, dtype):
    x, w = _gradient(rows, cols, dtype), ref.make(5)((rows, cols), dtype)
    want = dg.orthogonalize(x, residual=w)
    for off, pad in ((1, 3), (3, 5), (8, 8)):
        x2, w2, out = (ref.pitched(t, cols + pad, off) for t in (x, w, w))
        got = dg.orthogonalize(x2, residual=w2, out=out)
        assert got.data_ptr() == out.data_ptr() and torch.equal(got, want)
        between = out.as_strided((rows - 1, pad), (cols + pad, 1), off + cols)
        assert bool(torch.isnan(between).all()), "written between the rows"


@pytest.mark.parametrize("m, extra", [(1, 0), (40, 60), (256, 0), (300, 700)])
def test_equal_singular_values_stay_equal(m, extra):
    """X = s I: every intermediate is a multiple of I, exactly zero elsewhere, and its size is off by
    one rounding of 2^-11 for each of at most 20 stored matrices, amplified by no more than 1.6 (the
    largest |p'(s)| s / p(s) on the way) ... a bound of 40 x 2^-11."""
    x = torch.zeros((m, m + extra), dtype=torch.float16, device="cuda")
    x.diagonal().fill_(0.01)
    got = dg.orthogonalize(x, out=torch.empty(x.shape, device="cuda"))
    want = nr.formula(x.double())
    assert torch.count_nonzero(got).item() == m
    d = got.diagonal().double()
    assert bool(((d / want.diagonal() - 1).abs() < 40 * 2.0 ** -11).all()), float((d / want.diagonal() - 1).abs().max())


def test_sizes_that_overflow_or_vanish_when_squared():
    """A power of two on X changes nothing where eps is 0, at the ends of bfloat16's range too."""
    x = _gradient(120, 500, torch.bfloat16, 4, 1.0)
    want = dg.orthogonalize(x, eps=0.0)
    for up in (2.0 ** 100, 2.0 ** 120, 2.0 ** -60, 2.0 ** -100):
        y = (x.double() * up).bfloat16()
        assert bool(torch.isfinite(y).all()) and torch.equal(y.double(), x.double() * up)
        assert torch.equal(dg.orthogonalize(y, eps=0.0), want), up


def test_eps_zeros_and_values_that_are_not_finite():
    x = _gradient(90, 200, torch.float32, 5, 1e-9)
    nr.check(dg.orthogonalize(x, eps=1e-7), x, eps=1e-7)  # eps is most of the divisor
    z = torch.zeros((90, 200), device="cuda")
    assert torch.count_nonzero(dg.orthogonalize(z)) == 0
    assert bool(torch.isnan(dg.orthogonalize(z, eps=0.0)).all())
    for bad in (float("nan"), float("inf"), float("-inf")):
        y = x.clone()
        y[3, 5] = bad
        assert bool(torch.isnan(dg.orthogonalize(y)).all())
    w = torch.ones((0, 5), device="cuda")
    assert dg.orthogonalize(w).shape == (0, 5) and dg.orthogonalize(w.t()).shape == (5, 0)


def test_rank_one():
    n = ref.make(6)
    x = (n((150, 1), torch.float32) @ n((1, 400), torch.float32)).to(torch.bfloat16)
    nr.check(dg.orthogonalize(x), x)


def test_overlapping_streams_and_graphs():
    xs = [_gradient(200, 700, torch.bfloat16, s) for s in (7, 8)]
    want = [dg.orthogonalize(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[dg.orthogonalize(x, stream=s) for _ in range(5)] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for gs, w in zip(got, want) for g in gs)
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(dg.orthogonalize(x))
        graphs.append(g)
    xs[0].copy_(xs[1])
    torch.cuda.synchronize()
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1]) and torch.equal(outs[1], want[1])


def test_a_wait_that_runs_out_is_reported(monkeypatch):
    import os

    x = _gradient(600, 900, torch.bfloat16)
    want = dg.orthogonalize(x, steps=1)
    torch.cuda.synchronize()
    monkeypatch.setenv("DGEMM_TC_TEST_STALL", "1")
    t0 = time.time()
    dg.orthogonalize(x, steps=1)
    torch.cuda.synchronize()
    elapsed = time.time() - t0
    monkeypatch.delenv("DGEMM_TC_TEST_STALL")
    st, where = dg.dgemm_watchdog_status(torch.cuda.current_stream().cuda_stream)
    csrc = os.path.join(os.path.dirname(os.path.abspath(dg.__file__)), "csrc")
    sites = {int(c, 16) for f in os.listdir(csrc) if f.startswith("newton")
             for c in re.findall(r"kSite\w+ = (0x[0-9a-f]+)", open(os.path.join(csrc, f), encoding="utf-8").read())}
    assert st == dg.ERR_WATCHDOG and where in sites, (st, hex(where))
    assert elapsed < 60
    assert torch.equal(dg.orthogonalize(x, steps=1), want)


def test_a_block_trained_with_orthogonalised_updates():
    """The use: a step's gradients of a feed-forward block, from the library, orthogonalised into its weights."""
    n = ref.make(13)
    D, F, M = 256, 704, 512
    x, dy = n((M, D), torch.bfloat16), n((M, D), torch.bfloat16, 0.05)
    w = [n(s, torch.bfloat16, s[0] ** -0.5) for s in ((D, F), (D, F), (F, D))]
    h, mean, rstd = dg.layer_norm(x, return_stats=True)
    _, g, u = dg.gated_ffn(h, *w, residual=x, return_saved=True)
    grads = dg.gated_ffn_backward(dy, h, *w, g, u)[1:]
    for p, grad in zip(w, grads):
        before = p.clone()
        lr = 0.02 * math.sqrt(max(1.0, p.shape[0] / p.shape[1]))
        dg.orthogonalize(grad, scale=-lr, residual=p, residual_scale=1 - 0.002, out=p)
        nr.check(p, grad, scale=-lr, residual=before, keep=1 - 0.002)


@pytest.mark.parametrize("shape", [(2048, 4096), (4096, 2048), (600, 1500)])
def test_updates_one_after_the_other(shape):
    """Matrices that alternate, larger together than L2, on one stream and on two at once: every
    result is the one of a call alone, to the last bit."""
    n = ref.make(shape[0])
    xs = [n(shape, torch.bfloat16) for _ in range(6)]
    rs = [n(shape, torch.float32) for _ in range(6)]
    want = []
    for x, r in zip(xs, rs):
        want.append(dg.orthogonalize(x, scale=-0.1, residual=r))
        torch.cuda.synchronize()
    for _ in range(3):
        got = [dg.orthogonalize(x, scale=-0.1, residual=r) for x, r in zip(xs, rs)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [dg.orthogonalize(x, scale=-0.1, residual=r, stream=streams[i % 3]) for i, (x, r) in enumerate(zip(xs, rs))]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("plan", [dict(TN=64, SPLITS=1), dict(TN=128, SPLITS=1)], ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("rows, cols", [(1, 1), (65, 64), (129, 200), (200, 129), (191, 193), (300, 700), (513, 520)])
def test_every_tile_gives_the_same(rows, cols, dtype, plan, monkeypatch):
    """Whatever the tiles, an element is the same sum in the same order of K."""
    x, r = _gradient(rows, cols, dtype), ref.make(5)((rows, cols), dtype)
    monkeypatch.setenv("DGEMM_NEWTON_PAIR", "0")
    monkeypatch.setenv("DGEMM_NEWTON_TN", "64")
    monkeypatch.setenv("DGEMM_NEWTON_SPLITS", "1")
    want = dg.orthogonalize(x, scale=0.5, residual=r)
    for k, v in plan.items():
        monkeypatch.setenv("DGEMM_NEWTON_" + k, str(v))
    assert torch.equal(dg.orthogonalize(x, scale=0.5, residual=r), want)
    assert torch.equal(dg.orthogonalize(x, scale=0.5, residual=r), want)
