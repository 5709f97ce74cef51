"""The gate gradient on CTA pairs, whose epilogue sends for its inputs a piece
ahead, when a wait of the kernel runs out: the call comes back, the status names
the site, and the same call gives the same bits afterwards."""
import pytest
import torch

import dense_gemm_f32_gb300 as dg
import gpu_util as gu
import ops_reference as ref
from test_gpu_fused_watchdog import _stalled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__

    __graft_entry__.build()
    yield
    gu.check_watchdog()


@pytest.mark.parametrize("M, D, F", [(2048, 256, 4096), (300, 64, 520)])
def test_inputs_sent_for_ahead(M, D, F, monkeypatch):
    """128 tiles for 76 pairs, and fewer tiles than pairs."""
    monkeypatch.setenv("DGEMM_FUSED_PAIR", "1")
    n = ref.make(9)
    bf = torch.bfloat16
    dy, x = n((M, D), bf, 0.2), n((M, D), bf)
    wg, wu, wd = n((D, F), bf, D ** -0.5), n((D, F), bf, D ** -0.5), n((F, D), bf, F ** -0.5)
    g, u = n((M, F), bf), n((M, F), bf)
    h, dgate, dup = (torch.zeros((M, F), dtype=bf, device="cuda") for _ in range(3))
    dwd = torch.zeros((F, D), dtype=bf, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def call():
        st = dg.dgemm_gated_ffn_backward(
            dg.DTYPE_BF16, dg.ACT_SILU, dg.OP_N, M, D, F, dy.data_ptr(), D, x.data_ptr(), D,
            wg.data_ptr(), F, wu.data_ptr(), F, wd.data_ptr(), D, g.data_ptr(), F, u.data_ptr(), F,
            h.data_ptr(), F, dgate.data_ptr(), F, dup.data_ptr(), F, 0, D, 0, F, 0, F,
            dwd.data_ptr(), D, stream)
        assert st == dg.OK

    call()
    want = [t.clone() for t in (h, dgate, dup, dwd)]
    d = [t.double() for t in (dy, x, wg, wu, wd, g, u)]
    ref.check(dwd, ref.gated_backward(*d, "silu", bf)[3], "dwd")
    for t in (h, dgate, dup, dwd):
        t.zero_()
    _stalled(call, "fused_pair.cu", monkeypatch)
    call()
    for t, w in zip((h, dgate, dup, dwd), want):
        assert torch.equal(t, w)
