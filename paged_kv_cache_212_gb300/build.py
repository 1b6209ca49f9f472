"""Build libpagedkv.so in-tree with nvcc for sm_103a (GB300).

Each .cu (device) and .cpp (host-only) translation unit compiles in parallel
to an object file, then one
link step produces the shared library (cudart linked statically, so the
library needs only the driver at run time).  Beside them g++ compiles the
native part of the Python binding (binding/native.cpp, against the installed
torch) into a CPython extension of its own, which the library does not need.
Rebuilds only when a source or header is newer than what was built from it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpagedkv.so")
NATIVE_SRC = os.path.join(HERE, "binding", "native.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedkv.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def native_lib() -> str:
    import torch
    return os.path.join(HERE, f"_native-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def native_up_to_date() -> bool:
    lib = native_lib()
    deps = [NATIVE_SRC, os.path.abspath(__file__)] + glob.glob(os.path.join(ROOT, "include", "*.h"))
    return os.path.exists(lib) and all(os.path.getmtime(p) <= os.path.getmtime(lib) for p in deps)


def build_native() -> str:
    """The binding's native part, for the torch that is installed."""
    import torch
    home = os.path.dirname(torch.__file__)
    lib, cuda = native_lib(), os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = lib + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{p}" for p in inc), NATIVE_SRC,
           "-o", tmp, f"-L{os.path.join(home, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {NATIVE_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def try_native(force: bool = False):
    """The binding's native part, where it is out of date.  The calls work without it, so
    what went wrong (no torch, no g++, errors) is returned; what an older source left is
    removed then, as it may not fit the library."""
    try:
        if force or not native_up_to_date():
            build_native()
        return None
    except Exception as e:
        try:
            os.remove(native_lib())
        except (ImportError, OSError):
            pass
        return e


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Builds what is out of date; the path of the library.  Raises where that cannot be
    built, and warns where the binding's native part cannot."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(try_native, force)
        if force or not up_to_date():
            build_library(verbose, ptxas_verbose)
        error = binding.result()
    if error is not None:
        warnings.warn(f"the native part of the binding was not built, its calls go through Python: {error!r}", RuntimeWarning)
    return LIB


def build_library(verbose: bool = False, ptxas_verbose: bool = False) -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    flags = ["-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
             "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [cc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose or ptxas_verbose:
        for _, err in results:
            if err.strip():
                print(err, file=sys.stderr)
    objs = [o for o, _ in results]
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
