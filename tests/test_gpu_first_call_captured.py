"""The first call of a process may be one that is captured: what the library makes once
(its scratch pool, a kernel's attributes) is made then."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys, torch
sys.path.insert(0, {root!r})
import dense_gemm_f32_gb300 as dg
gen = torch.Generator(device="cuda").manual_seed(1)
def n(*s): return torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
x, w, u, r = n(40, 200), n(200, 333), n(200, 333), n(40, 200)
q = torch.randint(-127, 128, (333, 201), generator=gen, dtype=torch.int8, device="cuda")[:, 1:]
s = torch.full((333,), 0.01, device="cuda")
calls = dict(
    columns=lambda: dg.quantize_int8(w, transpose=True)[0],
    rows=lambda: dg.quantize_int8(w)[0],
    linear=lambda: dg.linear_int8(x, q, s),
    few=lambda: dg.linear_int8(x[:2], q, s),
    block=lambda: dg.gated_ffn_int8(x, q, s, q, s, q.t().contiguous(), s[:200], residual=r),
    update=lambda: dg.orthogonalize(w, residual=u))
call = calls[{name!r}]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = call()
for _ in range(3):
    g.replay()
torch.cuda.synchronize()
assert torch.equal(out, call()), "the replay and the call differ"
"""


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["columns", "rows", "linear", "few", "block", "update"])
def test_first_call_is_captured(name):
    import __graft_entry__

    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=ROOT, name=name)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
