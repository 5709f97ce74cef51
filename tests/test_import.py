"""The package's C entry points need no PyTorch: it is imported by the calls that
take tensors, not by the package."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BLOCKED = """
import importlib.abc, sys
class Block(importlib.abc.MetaPathFinder):
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ImportError("no PyTorch here")
sys.meta_path.insert(0, Block())
"""


def _python(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.strip()


def test_c_entry_points_without_pytorch():
    from dense_gemm_f32_gb300 import build

    build.build()
    out = _python(BLOCKED + """
import dense_gemm_f32_gb300 as dg
assert dg.dgemm_linear(dg.DTYPE_F32, 0, 0, 1, 1, 1, 0, 1, 0, 1, 0, 0, 1, 0, 1, 0, 1) == dg.ERR_UNSUPPORTED
print(dg.dgemm_status_string(dg.OK), callable(dg.linear), callable(dg.matmul))
""")
    assert out == "success True True"


def test_the_import_alone_does_not_bring_pytorch_in():
    assert _python("import sys, dense_gemm_f32_gb300; print('torch' in sys.modules)") == "False"
