"""Builds libsparseattn.so in-tree with nvcc for sm_100a.

``python -m long_context_mean_b200.build`` compiles every ``csrc/*.cu`` into
an object (in parallel, only when a source or header is newer than its
object) and links them into ``long_context_mean_b200/libsparseattn.so``.
The CUDA runtime is linked statically; no libcuda link is needed (driver
entry points are fetched at run time).  ``csrc/binding.cpp`` becomes
``_serve.so``, the compiled Python binding of the serving operators; it alone
needs torch, the Python headers and g++, and without them only it is left out.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsparseattn.so")
BINDING = os.path.join(PKG, "_serve.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsparseattn.so")
    return exe


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src: str, extra: list[str], verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), _newest_header()):
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr, flush=True)
    return obj


def _binding_world() -> str:
    """The interpreter and the torch that a binding is built for, and works with."""
    import importlib.metadata
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "none"
    return f"{sys.implementation.cache_tag} torch {torch}"


class BindingUnavailable(RuntimeError):
    """What the Python binding is built with is not there (the C library needs none of it)."""


def build_binding(verbose: bool = False) -> str:
    """The compiled Python binding of the serving operators (csrc/binding.cpp, host code against torch's headers)."""
    src = os.path.join(CSRC, "binding.cpp")
    stamp, world = os.path.join(BUILD, "_serve.stamp"), _binding_world()
    if os.path.exists(BINDING) and os.path.getmtime(BINDING) >= max(os.path.getmtime(src), _newest_header()):
        if os.path.exists(stamp) and open(stamp).read() == world:
            return BINDING
    import sysconfig

    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError as e:
        raise BindingUnavailable(f"torch cannot be imported: {e}") from e
    if shutil.which("g++") is None:
        raise BindingUnavailable("g++ not found")
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], INCLUDE,
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    for header in ("Python.h", "torch/csrc/utils/pybind.h", "cuda_runtime_api.h"):
        if not any(os.path.exists(os.path.join(d, header)) for d in inc):
            raise BindingUnavailable(f"the header {header} was not found")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-DTORCH_EXTENSION_NAME=_serve", f'-DBUILT_FOR_TORCH="{torch.__version__}"', *[x for d in inc for x in ("-isystem", d)], src, "-o", BINDING + ".tmp",
           "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(BINDING + ".tmp", BINDING)
    with open(stamp, "w") as f:
        f.write(world)
    return BINDING


def build(verbose: bool = False, extra: list[str] | None = None, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    extra = list(extra or [])
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for s in srcs:
            o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
            if os.path.exists(o):
                os.remove(o)
    if force and os.path.exists(BINDING):
        os.remove(BINDING)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(build_binding, verbose)
        objs = list(ex.map(lambda s: _compile(s, extra, verbose), srcs))
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [nvcc(), *ARCH, "-shared", "-o", LIB + ".tmp", *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(LIB + ".tmp", LIB)
    try:
        binding.result()
    except BindingUnavailable as e:
        warnings.warn(f"libsparseattn.so is built, its Python binding of the serving operators is not: {e}", stacklevel=2)
    return LIB


if __name__ == "__main__":
    args = sys.argv[1:]
    xtra = [a for a in args if a not in ("-v", "--force")]
    print(build(verbose="-v" in args, extra=xtra, force="--force" in args))
