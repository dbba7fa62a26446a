"""Build libnorm.so in-tree: nvcc for sm_103a, one object per translation
unit compiled in parallel, static CUDA runtime, no cmake. Next to it
_binding.so, the native half of the Python binding of the group norm, gradient,
head norm and dropout calls (g++ against the installed torch's headers, linked with
libnorm.so); where that does not build, the rest does."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnorm.so")
NATIVE_SRC = os.path.join(PKG, "native", "binding.cpp")
NATIVE = os.path.join(PKG, "_binding.so")
NATIVE_KEY = os.path.join(BUILD, "binding.key")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libnorm")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _library_up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _native_key() -> str:
    """What _binding.so is compiled against, beyond its sources."""
    import platform
    import sys

    import torch

    return "\n".join((sys.implementation.cache_tag, platform.machine(), torch.__version__, torch.__file__))


def native_matches() -> bool:
    """Whether _binding.so was compiled against this torch and interpreter
    (unknown without its key: yes)."""
    try:
        with open(NATIVE_KEY) as f:
            return f.read() == _native_key()
    except FileNotFoundError:
        return True


def _native_up_to_date() -> bool:
    if not os.path.exists(NATIVE) or not os.path.exists(NATIVE_KEY) or not native_matches():
        return False
    t = os.path.getmtime(NATIVE)
    return all(os.path.getmtime(p) <= t for p in [NATIVE_SRC, *glob.glob(os.path.join(INCLUDE, "*.h"))])


def up_to_date() -> bool:
    return _library_up_to_date() and _native_up_to_date()


def _compile_native() -> str:
    """The object file of the native binding."""
    import sysconfig

    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, "binding.o")
    # -isystem: the headers' own warnings are theirs
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", f"-I{INCLUDE}", "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"], "-isystem", cuda,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-c", NATIVE_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {NATIVE_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_native(obj: str) -> None:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = NATIVE + f".tmp{os.getpid()}"
    # the CUDA runtime the binding asks for the SM count is libnorm's kind: static
    cudart = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "lib64")
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libnorm.so", "-Wl,-rpath,$ORIGIN", f"-L{lib}",
           "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}", f"-L{cudart}",
           "-lcudart_static", "-ldl", "-lrt", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)


def _build_library(verbose: bool, extra_flags: list[str]) -> None:
    cc = nvcc()
    flags = NVCC_FLAGS + extra_flags

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(sources()), os.cpu_count() or 4))) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    library, native = force or not _library_up_to_date(), force or not _native_up_to_date()
    if not library and not native:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_native) if native else None
        if library:
            _build_library(verbose, extra_flags or [])
        if native:
            try:
                _link_native(obj.result())
                with open(NATIVE_KEY, "w") as f:
                    f.write(_native_key())
            except Exception as e:
                # libnorm.so and the calls through ctypes do without it; those that need it say that it is missing
                for p in (NATIVE, NATIVE_KEY):
                    if os.path.exists(p):
                        os.remove(p)
                warnings.warn(f"libnorm.so is built, but not _binding.so, which the group norm and gradient calls need: {e}",
                              RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
