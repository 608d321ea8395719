"""Build libk8v4.so in-tree for sm_103a: one nvcc process per translation unit,
run in parallel, then one shared link; and the extension module of the Python
binding beside it.  Used by __graft_entry__.build()."""
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
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libk8v4.so")
BINDING = os.path.join(BUILD, "_k8v4_binding.so")
BINDING_ERROR = os.path.join(BUILD, "binding_error.log")      # why the module could not be built, if so
SOURCES = ["k8v4_api.cu", "k8v4_append.cu", "k8v4_attend.cu", "k8v4_decode.cu", "k8v4_verify.cu", "k8v4_combine.cu", "k8v4_prefill.cu", "k8v4_noalloc.cu",
           "k8v4_stream.cu", "k8v4_rope.cu", "k8v4_append_rope.cu", "k8v4_accept.cu", "k8v4_shared.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the k8v4 CUDA library cannot be built")
    return cand


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _binding_tag() -> str:
    """What the extension module is compiled against: another torch or Python has other C++ symbols."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def binding_built() -> bool:
    """Whether the extension module is there, for this torch and Python."""
    if not os.path.exists(BINDING) or not os.path.exists(BINDING + ".tag"):
        return False
    with open(BINDING + ".tag") as f:
        return f.read() == _binding_tag()


def _compile_binding() -> str | None:
    """Build the extension module that checks tensors for the calls of csrc/k8v4_binding.cpp.
    Returns why it could not be built (no Python headers, a torch whose headers do not
    compile, ...), or None."""
    tmp = BINDING + f".tmp{os.getpid()}"
    try:
        import torch
        base = os.path.dirname(torch.__file__)
        inc = [os.path.join(base, "include"), sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
        cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{d}" for d in inc],
               os.path.join(CSRC, "k8v4_binding.cpp"), "-o", tmp, f"-L{os.path.join(base, 'lib')}", "-ltorch_python",
               "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            return f"g++ failed on k8v4_binding.cpp:\n{r.stdout}\n{r.stderr}"
        if os.path.exists(BINDING + ".tag"):
            os.remove(BINDING + ".tag")
        os.replace(tmp, BINDING)
        with open(BINDING + ".tag", "w") as f:
            f.write(_binding_tag())
        return None
    except (ImportError, OSError, RuntimeError) as e:
        return f"k8v4_binding.cpp could not be compiled: {e}"


def _stale(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(HERE, "..", "include", "k8v4.h"))
    deps.append(__file__)
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _build_library(ex: cf.Executor, verbose: bool) -> None:
    results = list(ex.map(_compile, SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for (_, log) in results:
            f.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is out of date.  The library needs nvcc alone: where the extension
    module cannot be built, that is a warning here and an error in the calls that use it."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding) if force or _stale(BINDING) or not binding_built() else None
        if force or _stale(LIB):
            _build_library(ex, verbose)
        failed = binding.result() if binding else None
    if binding and os.path.exists(BINDING_ERROR):
        os.remove(BINDING_ERROR)
    if failed:
        if os.path.exists(BINDING):         # of older sources, or for another torch
            os.remove(BINDING)
        with open(BINDING_ERROR, "w") as f:
            f.write(failed)
        warnings.warn(f"libk8v4.so is built, its extension module is not: {failed}")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
