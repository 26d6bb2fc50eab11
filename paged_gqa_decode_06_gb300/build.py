"""Builds libpaged_gqa_decode.so in-tree (``_build/``) with nvcc for sm_103a.

Each .cu translation unit compiles in its own nvcc process, in parallel; the
objects are linked into one shared library whose only dependencies are the C
and C++ runtimes (cudart is linked statically and reaches the driver at run
time), so it loads on a machine without a GPU.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB_NAME = "libpaged_gqa_decode.so"
LIB_PATH = os.path.join(BUILD, LIB_NAME)
# The checked build (-DPGD_CHECKED): every global index and TMA coordinate of
# the kernels is range-checked; a violation raises DECODE_ATTN_DEV_CHECK and
# skips the access.  A stand-in for a memory checker, for tests on small
# cases; selected at load time with DECODE_ATTN_CHECKED=1.
BUILD_CHECKED = os.path.join(HERE, "_build_checked")
LIB_CHECKED_NAME = "libpaged_gqa_decode_checked.so"
LIB_CHECKED_PATH = os.path.join(BUILD_CHECKED, LIB_CHECKED_NAME)


def binding_path() -> str:
    """The Python binding's quick way (csrc/binding.cpp), one module for both builds.
    It is compiled against one torch's classes and one Python's objects, so its name
    carries both: another does not load it."""
    import torch
    return os.path.join(BUILD, f"_binding-{torch.__version__}"
                               f"{sysconfig.get_config_var('EXT_SUFFIX') or '.so'}")


def checked_requested() -> bool:
    return os.environ.get("DECODE_ATTN_CHECKED") == "1"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return ([f for f in glob.glob(os.path.join(CSRC, "*")) if not f.endswith(".cpp")] +
            [os.path.join(os.path.dirname(HERE), "include", "decode_attn.h")])


def _up_to_date(lib: str, deps=None) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in (deps or _deps()))


def _compile(src: str, out_dir: str, extra: tuple) -> tuple[str, str]:
    obj = os.path.join(out_dir, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    with open(obj + ".ptxas.txt", "w") as f:  # register / spill / smem report
        f.write(r.stderr)
    return obj, r.stderr


def build_binding(force: bool = False):
    """Compile csrc/binding.cpp against the installed torch; None (and a warning)
    where that cannot be done: the binding then takes its Python way."""
    src = os.path.join(CSRC, "binding.cpp")
    header = os.path.join(os.path.dirname(HERE), "include", "decode_attn.h")
    try:
        import torch
        from torch.utils.cpp_extension import include_paths, library_paths
    except ImportError:
        return None
    path = binding_path()
    if not force and _up_to_date(path, [src, header]):
        return path
    tmp = path + f".tmp{os.getpid()}"
    abi = int(getattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", True))
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
           *["-I" + p for p in [*include_paths(), sysconfig.get_paths()["include"]]], src, "-o",
           tmp, *["-L" + p for p in library_paths()], "-lc10", "-ltorch_cpu", "-ltorch_python"]
    error = ""
    try:
        os.makedirs(BUILD, exist_ok=True)
        if os.path.exists(path):  # (of other sources: not loaded if this build fails)
            os.remove(path)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            error = r.stderr
        else:
            os.replace(tmp, path)
    except OSError as e:
        error = str(e)
    if error:
        warnings.warn(f"the quick binding was not built, calls take the Python way:\n{error}")
        return None
    return path


def build(force: bool = False, verbose: bool = False, checked=None) -> str:
    """Compile every .cu under csrc/ and link the shared library (the checked
    build when ``checked``, by default when DECODE_ATTN_CHECKED=1)."""
    if checked is None:
        checked = checked_requested()
    out_dir, lib = (BUILD_CHECKED, LIB_CHECKED_PATH) if checked else (BUILD, LIB_PATH)
    extra = ("-DPGD_CHECKED",) if checked else ()
    os.makedirs(out_dir, exist_ok=True)
    if not force and _up_to_date(lib):
        build_binding()
        return lib
    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        binding = ex.submit(build_binding, force)
        results = list(ex.map(lambda s: _compile(s, out_dir, extra), srcs))
        binding.result()  # (raises what it raised)
    if verbose:
        for _, log in results:
            print(log)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose=True))
