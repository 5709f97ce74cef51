"""Build libdgemm.so (the C-ABI library) in-tree with nvcc for sm_103a, and
beside it _torch_binding.so (the operators' tensor calls) with the host
compiler against the installed PyTorch.

The translation units compile in parallel; the link keeps only the symbols
declared in include/dgemm.h visible.  ptxas resource usage (-Xptxas -v:
registers, spills, shared memory per kernel) is written to
_build/ptxas_<unit>.log next to the objects.
"""
import concurrent.futures as cf
import importlib.util
import os
import platform
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdgemm.so")
BINDING = os.path.join(PKG, "_torch_binding.so")
HEADER = os.path.join(ROOT, "include", "dgemm.h")
BINDING_SOURCE = "torch_binding.cpp"
# (source, object name, defines): simt.cu and tc.cu are compiled once per
# operand layout so that the four layouts build in parallel.
UNITS = ([("api.cu", "api", []), ("staging.cu", "staging", []), ("ops_api.cu", "ops_api", []),
          ("norm.cu", "norm", []), ("rowops.cu", "rowops", []),
          ("fused.cu", "fused", []), ("quant.cu", "quant", []), ("int8.cu", "int8", []),
          ("int8_small.cu", "int8_small", []), ("int8_pair.cu", "int8_pair", []), ("int8_row.cu", "int8_row", []), ("newton.cu", "newton", []),
          ("newton_pair.cu", "newton_pair", []), ("newton_small.cu", "newton_small", [])]
         + [("fused_pair.cu", f"fused_pair_{u}", [f"-DDGEMM_FUSED_UNIT={u}"]) for u in range(3)]
         + [("fused_small.cu", f"fused_small_{u}", [f"-DDGEMM_FUSED_UNIT={u}"]) for u in range(4)]
         + [("simt.cu", f"simt_{u}", [f"-DDGEMM_SIMT_UNIT={u}"]) for u in range(4)]
         + [("tc.cu", f"tc_{u}", [f"-DDGEMM_TC_UNIT={u}"]) for u in range(4)])
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
EXPORTS = ["gemm_f32_simt", "gemm_f32_tc", "gemm_bf16_tc", "dgemm_status_string",
           "dgemm_last_cuda_error", "dgemm_watchdog_status", "dgemm_version",
           "dgemm_kernel_launches", "gemm_f32_tc_noalloc", "gemm_f16_tc", "dgemm_gemm_ex",
           "gemm_f8_tc", "dgemm_layer_norm", "dgemm_layer_norm_backward", "dgemm_linear",
           "dgemm_linear_backward", "dgemm_gated_ffn", "dgemm_gated_ffn_backward",
           "dgemm_quantize_int8", "dgemm_linear_int8_workspace", "dgemm_linear_int8",
           "dgemm_gated_ffn_int8_workspace", "dgemm_gated_ffn_int8",
           "dgemm_orthogonalize_workspace", "dgemm_orthogonalize"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdgemm.so")


def _newer(path, sources):
    """Whether a source is newer than the built file, or there is none."""
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(s) > t for s in sources if os.path.isfile(s))


def _library_stale():
    sources = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != BINDING_SOURCE]
    return _newer(LIB, sources + [HEADER, __file__])


def binding_key():
    """The PyTorch, Python and machine that the tensor calls are compiled for; they are C++ against
    PyTorch's own types and do not serve another.  None without PyTorch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    with open(os.path.join(os.path.dirname(spec.origin), "version.py"), encoding="utf-8") as f:
        version = re.search(r"^__version__ = ['\"]([^'\"]+)", f.read(), re.M)
    return f"PyTorch {version and version.group(1)}, Python {sys.implementation.cache_tag}, {platform.machine()}"


def built_key(binding):
    """The key that a built file of the tensor calls has beside it, or None."""
    try:
        with open(binding + ".key", encoding="utf-8") as f:
            return f.read()
    except OSError:
        return None


def binding_stale():
    return (_newer(BINDING, [os.path.join(CSRC, BINDING_SOURCE), HEADER, __file__])
            or built_key(BINDING) != binding_key())


def _run(cmd, what):
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{what}: {cmd[0]}: {e.strerror}") from e
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stderr[-6000:]}")
    return r.stdout + r.stderr


def _compile_binding(nvcc):
    """The tensor calls' object file, and the directory of PyTorch's libraries."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("the tensor calls need PyTorch, which is not installed")
    torch = os.path.dirname(spec.origin)
    obj = os.path.join(BUILD, "torch_binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    include = os.path.join(torch, "include")
    _run([os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden",
          "-isystem", include,
          "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
          "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj],
         "the host compiler failed on the tensor calls")
    return obj, os.path.join(torch, "lib")


def _link_binding(obj, torch_lib):
    tmp = BINDING + f".tmp{os.getpid()}"
    _run([os.environ.get("CXX", "g++"), "-shared", obj, "-o", tmp, LIB, "-L", torch_lib,
          "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10",
          "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"], "link of the tensor calls failed")
    if os.path.exists(BINDING + ".key"):
        os.remove(BINDING + ".key")  # never the new key beside the old file
    os.replace(tmp, BINDING)
    with open(BINDING + ".key", "w", encoding="utf-8") as f:
        f.write(binding_key())


def _compile(nvcc, unit):
    source, name, defines = unit
    src = os.path.join(CSRC, source)
    obj = os.path.join(BUILD, name + ".o")
    cmd = [nvcc, *ARCH, "-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC",
           "-Xptxas", "-v", *defines, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(BUILD, f"ptxas_{name}.log"), "w") as f:
        f.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {name}:\n{r.stderr[-6000:]}")
    return obj


def _link_library(nvcc, objs):
    vs = os.path.join(BUILD, "exports.map")
    with open(vs, "w") as f:
        f.write("{\n  global:\n" + "".join(f"    {s};\n" for s in EXPORTS) + "  local: *;\n};\n")
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-Xlinker", "-soname=libdgemm.so", "-Xlinker",
          f"--version-script={vs}", *objs, "-o", tmp], "link failed")
    os.replace(tmp, LIB)


def _build(force, library, binding):
    """Build what is asked for and stale, in parallel.  Returns why the tensor calls could not be
    built, or None; the library never waits for them."""
    library, binding = library and (force or _library_stale()), binding and (force or binding_stale())
    if not library and not binding:
        return None
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    with cf.ThreadPoolExecutor(max_workers=min(len(UNITS) + 1, os.cpu_count() or 4)) as ex:
        compiled = ex.submit(_compile_binding, nvcc) if binding else None
        if library:
            _link_library(nvcc, list(ex.map(lambda u: _compile(nvcc, u), UNITS)))
        try:
            if compiled is not None:
                _link_binding(*compiled.result())
        except RuntimeError as e:
            return str(e)
    return None


def build_library(force=False):
    """Compile libdgemm.so (if stale) and return its path; needs no PyTorch."""
    _build(force, True, False)
    return LIB


def build_binding(force=False):
    """Compile the tensor calls (if stale), and the library that they call, and return their path."""
    why = _build(force, True, True)
    if why is not None:
        raise RuntimeError(f"the operators' tensor calls were not built: {why}")
    return BINDING


def build(force=False, verbose=False):
    """Compile (if stale) the library and the tensor calls, and return the path of libdgemm.so.
    Where the tensor calls cannot be built (no PyTorch, say), that is reported and the library
    serves without them."""
    why = _build(force, True, True)
    if why is not None:
        print(f"the operators' tensor calls were not built: {why}", file=sys.stderr)
    if verbose:
        for _, name, _ in UNITS:
            with open(os.path.join(BUILD, f"ptxas_{name}.log")) as f:
                sys.stdout.write(f.read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
