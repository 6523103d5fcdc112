"""In-tree build of ``libkda.so`` (sm_103a) with plain nvcc, and of the Python
extension ``_layer_calls.so`` with the host compiler.

Each ``csrc/*.cu`` translation unit is compiled in parallel to an object
(``-gencode arch=compute_103a,code=sm_103a -lineinfo -O3``), then the objects
are linked into ``chunked_gated_delta_gb300/libkda.so``.  The extension
(``csrc_torch/layer_calls.cpp``: the Python calls of the served layer's
operators, on torch's tensors) is compiled beside them against torch's headers
and linked to the library.  The build is skipped when both are newer than every
source and header, and the extension is this interpreter's and its torch's.  The
library does not need torch: without it only the library is built, and an
extension that fails to compile is reported after the library is there.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
CSRC_TORCH = os.path.join(PKG, "csrc_torch", "layer_calls.cpp")
LIB = os.path.join(PKG, "libkda.so")
EXTENSION = os.path.join(PKG, "_layer_calls.so")
OBJDIR = os.path.join(PKG, "_build")
# What the extension was built against: it reads torch's C++ objects, whose layout is its version's own.
BUILT_FOR = os.path.join(OBJDIR, "layer_calls.built_for")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I" + INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the KDA CUDA library cannot be built")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [CSRC_TORCH, os.path.abspath(__file__)])


def _have_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def _interpreter() -> str:
    """This interpreter and its torch."""
    import torch
    return f"torch {torch.__version__} in {os.path.dirname(torch.__file__)}, Python {sysconfig.get_config_var('SOABI')}\n"


def extension_matches() -> bool:
    """Whether the extension was built for this interpreter and its torch."""
    try:
        with open(BUILT_FOR) as f:
            return f.read() == _interpreter()
    except OSError:
        return False


def up_to_date() -> bool:
    built = [LIB, EXTENSION] if _have_torch() else [LIB]
    if not all(os.path.exists(p) for p in built) or (len(built) > 1 and not extension_matches()):
        return False
    t = min(os.path.getmtime(p) for p in built)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r


def _host_compiler() -> str:
    for cand in (os.environ.get("CXX"), "g++", "c++"):
        if cand and shutil.which(cand):
            return cand
    raise RuntimeError("no C++ compiler found: the Python extension cannot be built")


def _compile_extension() -> str:
    """csrc_torch/layer_calls.cpp to an object, against this interpreter's torch."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    obj = os.path.join(OBJDIR, "layer_calls.cpp.o")
    _run([_host_compiler(), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + sysconfig.get_paths()["include"],
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
          "-c", CSRC_TORCH, "-o", obj], "compiling layer_calls.cpp")
    return obj


def _link_extension(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = EXTENSION + f".tmp{os.getpid()}"
    _run([_host_compiler(), "-shared", "-o", tmp, obj, "-L" + PKG, "-l:" + os.path.basename(LIB), "-L" + lib,
          "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN:" + lib],
         "linking the Python extension")
    if os.path.exists(BUILT_FOR):
        os.remove(BUILT_FOR)
    os.replace(tmp, EXTENSION)
    with open(BUILT_FOR, "w") as f:
        f.write(_interpreter())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libkda.so and the Python extension; returns the library's path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = sources()

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        extension = ex.submit(_compile_extension) if _have_torch() else None
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of libkda.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if extension is not None:
        _link_extension(extension.result())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
