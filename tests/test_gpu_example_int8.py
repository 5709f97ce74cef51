"""The feed-forward example with orthogonalised updates and 8-bit serving: that it runs, and that
what it serves in 8 bits is what it trained."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location(
        "feed_forward_block", os.path.join(ROOT, "examples", "feed_forward_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("width, hidden, outputs, tokens", [(256, 704, 96, 512), (200, 333, 65, 301)])
def test_update_then_serve(example, width, hidden, outputs, tokens):
    import dense_gemm_f32_gb300 as dg

    model = example.FeedForward(width, hidden, outputs, seed=4)
    x = torch.randn((tokens, width), device="cuda").to(torch.bfloat16)
    target = torch.randn((tokens, outputs), device="cuda")
    before = {k: v.clone() for k, v in model.master.items()}
    for _ in range(3):
        loss = model.step(x, target, 0.05, orthogonal_lr=0.02)
    assert bool(torch.isfinite(loss))
    for k, v in model.master.items():
        assert bool(torch.isfinite(v).all()) and not torch.equal(v, before[k])
    # no singular value of an update is much above 1: a p(x) of x in [0, 1] is at most 1.21
    w = model.master["w_gate"]
    m = model.momentum["w_gate"]
    s = torch.linalg.svdvals((dg.orthogonalize(m, scale=-0.02, residual=w) - w).double() / 0.02)
    assert s[0] < 1.3
    q = model.quantised()
    full, served = model.forward(x).double(), model.forward_int8(x, q).double()
    single = torch.stack([model.forward_int8(x[i], q) for i in range(4)]).double()
    # rows in 8 bits are off by half a step, 1 / 254 of the row's top: about 1 percent of a
    # product's norm, three products one behind the other and both operands of each
    assert ((served - full).norm() / full.norm()).item() < 0.06
    # a token alone and in the batch: bf16 results half a step apart, here and there an integer
    assert ((single - served[:4]).norm() / served[:4].norm()).item() < 0.02
