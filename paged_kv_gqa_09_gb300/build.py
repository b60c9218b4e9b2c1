"""Build libpkv.so (the CUDA kernels and the C ABI) for sm_103a, in-tree.

Each ``csrc/*.cu`` is compiled to an object in parallel by nvcc and linked
into ``paged_kv_gqa_09_gb300/_build/libpkv.so``; beside it the host compiler
builds ``_pkv_call.so`` from ``csrc/binding.cpp`` against the running Python
and PyTorch.  Runs on a machine without a GPU (nvcc cross-compiles).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libpkv.so")
CALL = os.path.join(OUT_DIR, "_pkv_call.so")
CALL_FOR = CALL + ".for"  # the Python and PyTorch it was compiled for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv")
    return path


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                   "-I", INCLUDE, "-I", CSRC, *extra]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "pkv.h")]


def _call_command(out: str) -> list[str]:
    import torch
    home = os.path.dirname(torch.__file__)
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    libs = os.path.join(home, "lib")
    return [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-shared", "-fPIC",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
            *[x for i in inc for x in ("-isystem", i)], os.path.join(CSRC, "binding.cpp"), "-o", out,
            "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def call_for() -> str:
    """What _pkv_call.so is compiled for: it reads tensors by this PyTorch's headers, through this Python's ABI."""
    import torch
    return f"{sysconfig.get_config_var('SOABI')} torch {torch.__version__} cxx11_abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def call_fits() -> bool:
    """Whether the built _pkv_call.so is for the running Python and PyTorch."""
    try:
        with open(CALL_FOR) as f:
            return f.read() == call_for()
    except OSError:
        return False


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(CALL) and call_fits()):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALL))
    return all(os.path.getmtime(f) <= t for f in [*_deps(), os.path.join(CSRC, "binding.cpp")])


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every kernel for sm_103a and link libpkv.so; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *_flags(extra), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    def compile_call():
        out = CALL + f".tmp{os.getpid()}"
        r = subprocess.run(_call_command(out), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"the host compiler failed on binding.cpp:\n{r.stderr}")
        return out

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        call = ex.submit(compile_call)
        results = list(ex.map(compile_one, _sources()))
        call_tmp = call.result()
    if verbose or ptxas_verbose:
        for _, err in results:
            if err:
                print(err)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart_static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if os.path.exists(CALL_FOR):  # it names nothing while the module changes
        os.remove(CALL_FOR)
    os.replace(call_tmp, CALL)
    with open(CALL_FOR + f".tmp{os.getpid()}", "w") as f:
        f.write(call_for())
    os.replace(f.name, CALL_FOR)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
