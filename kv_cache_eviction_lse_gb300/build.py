"""Build the kvs CUDA library in-tree: kv_cache_eviction_lse_gb300/_lib/libkvs.so, and beside
it kvs_binding.so, the Python side of the calls made for every token.

Every CUDA translation unit is compiled for sm_103a only (one -gencode), in parallel, then
linked into one shared library with the CUDA runtime linked statically.  The binding is plain
C++ against the headers of the Python and torch that run the build; it is built anew for
others.  Where it cannot be built (no g++, no headers) the library is built all the same, with
a warning: only the serving calls need the binding, and they say so.

    python -m kv_cache_eviction_lse_gb300.build          # build (incremental)
    python -m kv_cache_eviction_lse_gb300.build --force  # rebuild everything
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT, "libkvs.so")
BINDING = os.path.join(OUT, "kvs_binding.so")
BUILT_FOR = os.path.join(OUT, "kvs_binding.txt")  # the Python and torch it was built for
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", f"-I{INCLUDE}"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the kvs CUDA library cannot be built")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "kvs.h"))
    return max(os.path.getmtime(f) for f in files)


def _run(what, cmd, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr, file=sys.stderr)


def hosts() -> str:
    """The Python and torch that a binding belongs to."""
    import torch
    return f"{sysconfig.get_config_var('SOABI')} torch {torch.__version__}"


def _fresh(*outputs) -> bool:
    newest = _deps_mtime()
    return all(os.path.exists(o) and os.path.getmtime(o) >= newest for o in outputs)


def _binding_object():
    import torch
    t = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    obj = os.path.join(OUT, "binding.cpp.o")
    _run("binding.cpp", ["g++", "-O2", "-std=c++17", "-fPIC", f"-I{t}",
                         f"-I{t}/torch/csrc/api/include", f"-I{cuda}",
                         f"-I{sysconfig.get_paths()['include']}",
                         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                         "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj])
    return obj


def _link_binding(obj):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    _run("link of the binding", ["g++", "-shared", "-o", tmp, obj, f"-L{OUT}", "-lkvs", f"-L{libs}",
                                 "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                                 "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, BINDING)
    with open(BUILT_FOR, "w") as f:
        f.write(hosts())


def _binding_fresh() -> bool:
    if not _fresh(BINDING) or not os.path.exists(BUILT_FOR):
        return False
    with open(BUILT_FOR) as f:
        return f.read() == hosts()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and return the path of libkvs.so."""
    os.makedirs(OUT, exist_ok=True)
    stale = force or not _fresh(LIB)
    try:
        binding_stale = stale or not _binding_fresh()
    except ImportError:  # no torch
        binding_stale = True
    if not stale and not binding_stale:
        return LIB
    if os.path.exists(BUILT_FOR):
        os.remove(BUILT_FOR)  # no binding of another library or Python is loaded meanwhile
    nvcc = _nvcc() if stale else None
    srcs = sources() if stale else []

    def compile_one(src):
        obj = os.path.join(OUT, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        _run(f"nvcc for {src}", cmd, verbose)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_binding_object)
        objs = list(ex.map(compile_one, srcs))
    if stale:
        tmp = LIB + ".tmp"
        _run("link", [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    try:
        _link_binding(binding.result())
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the binding of the serving calls was not built: {e}", stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
