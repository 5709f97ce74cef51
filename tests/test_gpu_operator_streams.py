"""Calls that overlap on two streams, from one host thread and from two, give what
they give alone.  Odd sizes: operands are staged and column sums joined, so every call
holds scratch that the other stream's must not touch."""
import threading

import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import ops_reference as ref

pytestmark = pytest.mark.gpu
M, D, F = 1000, 1013, 997
CALLS = 40


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()


def _work(seed):
    """The operators' calls on inputs of this seed, as functions of a stream."""
    n, bf = ref.make(seed), torch.bfloat16
    x, dy, dd = n((M, D), bf), n((M, D), bf, 0.2), n((M, F), bf, 0.2)
    ws = [n((D, F), bf, 0.03), n((D, F), bf, 0.03), n((F, D), bf, 0.03)]
    g, u, z = n((M, F), bf), n((M, F), bf), n((M, F), bf)
    w, b = n((D,), bf), n((F,), bf)
    _, mean, rstd = dg.layer_norm(x, w, w, return_stats=True)
    return [lambda s: [dg.linear(x, ws[0], b, "gelu", z, stream=s)],
            lambda s: [t for t in dg.linear_backward(dd, x, ws[0], "silu", z, stream=s)],
            lambda s: [dg.gated_ffn(x, *ws, residual=dy, stream=s)],
            lambda s: [t for t in dg.gated_ffn_backward(dy, x, *ws, g, u, stream=s)],
            lambda s: [t for t in dg.layer_norm_backward(dy, x, w, mean, rstd, dresidual=x, stream=s)]]


def _alone(work):
    want = [call(None) for call in work]
    torch.cuda.synchronize()
    return want


def _enqueue(work, stream, out):
    for i in range(CALLS):
        out.append((i % len(work), work[i % len(work)](stream)))


def _same(out, want):
    assert len(out) == CALLS
    for at, got in out:
        assert all(torch.equal(a, b) for a, b in zip(got, want[at])), f"call {at} differs"


@pytest.mark.parametrize("threads", [False, True])
def test_two_streams_at_once(threads):
    work = [_work(1), _work(2)]
    want = [_alone(w) for w in work]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        out = [[], []]
        if threads:
            pair = [threading.Thread(target=_enqueue, args=(w, s, o)) for w, s, o in zip(work, streams, out)]
            for t in pair:
                t.start()
            for t in pair:
                t.join()
        else:  # taking turns, so that both queues are never empty
            for i in range(CALLS):
                for w, s, o in zip(work, streams, out):
                    o.append((i % len(w), w[i % len(w)](s)))
        torch.cuda.synchronize()
        for o, w in zip(out, want):
            _same(o, w)
    gu.check_watchdog()
