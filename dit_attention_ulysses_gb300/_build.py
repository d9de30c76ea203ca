"""Build libxsattn.so (the sm_103a kernels + C ABI) in-tree with nvcc.

The translation units are compiled in parallel and linked into one shared
library next to this file.  Only nvcc and the CUDA runtime are needed; no
PyTorch headers are involved (the C ABI takes plain pointers).

Beside it, where Python's and PyTorch's headers are there, g++ compiles the
binding of the serving calls (_binding.so, csrc/binding.cpp); without it their
arguments are checked in Python.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
SOURCES = ["attn_fwd.cu", "attn_paged.cu", "attn_paged8.cu", "attn_paged8_rows.cu", "attn_paged_rows.cu", "paged_plan.cu", "paged_step.cu", "rope.cu", "relayout.cu",
           "burst_gap.cu", "paged8.cu", "api.cu", "api_paged.cu", "api_paged8.cu"]
HEADERS = ["kernels.h", "host.h", "paged.h", "paged_host.h", "rope_tile.cuh", "codes8.cuh", "paged_walk.cuh", "paged_chunk.cuh", "paged_rows.cuh", "attn_tile.cuh", "device_wait.cuh", "error_words.cuh", "ptx.cuh", os.path.join("..", "..", "include", "xsattn.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.isdir(home):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _nvcc() -> str:
    return os.path.join(cuda_home(), "bin", "nvcc")


# Library variants: the product library, and a build with per-tile timestamps
# (XS_TILE_SPANS; read by dit_attention_ulysses_gb300.spans) for measurements.
VARIANTS = {"": ([], "libxsattn.so", "_build"), "spans": (["-DXS_TILE_SPANS"], "libxsattn_spans.so", "_build_spans")}


def lib_path(variant: str = "") -> str:
    return os.path.join(HERE, VARIANTS[variant][1])


def _stale(lib: str) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, s) for s in SOURCES + HEADERS] + [__file__]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


BINDING = os.path.join(HERE, "_binding.so")


def _binding_headers() -> str | None:
    """PyTorch's directory, if its headers and Python's are installed."""
    spec = importlib.util.find_spec("torch")
    torch_dir = os.path.dirname(spec.origin) if spec and spec.origin else ""
    found = [os.path.join(torch_dir, "include", "torch", "csrc", "autograd", "python_variable.h"),
             os.path.join(sysconfig.get_paths()["include"], "Python.h")]
    return torch_dir if torch_dir and all(map(os.path.exists, found)) and shutil.which("g++") else None


def build_binding(force: bool = False) -> str | None:
    """Compile the binding (if stale) and return its path; None without the headers, or if this
    PyTorch does not compile it."""
    torch_dir = _binding_headers()
    if torch_dir is None:
        return None
    src = os.path.join(CSRC, "binding.cpp")
    deps = [src, os.path.join(CSRC, "..", "..", "include", "xsattn.h"), __file__,
            os.path.join(torch_dir, "version.py")]
    if not force and os.path.exists(BINDING) and all(os.path.getmtime(d) <= os.path.getmtime(BINDING) for d in deps
                                                     if os.path.exists(d)):
        return BINDING
    inc, lib = os.path.join(torch_dir, "include"), os.path.join(torch_dir, "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w", src, "-o", tmp]
    for d in (inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
              os.path.join(cuda_home(), "include")):
        cmd += ["-I", d]
    cmd += ["-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:   # the library works without it
        warnings.warn(f"binding.cpp was not compiled; serving calls check their arguments in Python:\n{r.stderr[-2000:]}")
        if os.path.exists(BINDING):
            os.remove(BINDING)
        return None
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, variant: str = "") -> str:
    """Compile (if stale) and return the path of libxsattn.so (or of a variant)."""
    defines, lib_name, build_dir = VARIANTS[variant]
    LIB = os.path.join(HERE, lib_name)
    if not force and not _stale(LIB):
        build_binding()
        return LIB
    bdir = os.path.join(HERE, build_dir)
    os.makedirs(bdir, exist_ok=True)
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-I", CSRC] + defines
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(bdir, src.replace(".cu", ".o"))
        cmd = [_nvcc(), "-c", os.path.join(CSRC, src), "-o", obj] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(build_binding, force)
        results = list(ex.map(compile_one, SOURCES))
        binding.result()
    if verbose:
        for _, log in results:
            if log:
                print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    libdir = os.path.join(cuda_home(), "lib64")
    cmd = [_nvcc(), "-shared", "-o", tmp] + [o for o, _ in results] + ARCH + [
        "--cudart", "shared", "-Xlinker", f"-rpath,{libdir}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv, variant="spans" if "spans" in sys.argv else ""))
