"""Builds the CUDA library ``libpaged_attn.so`` in-tree for sm_103a.

Each ``csrc/*.cu`` file is compiled by nvcc in parallel, then linked into one
shared library next to this file (``lib/libpaged_attn.so``).  Beside it
``csrc/native_binding.cpp``, the Python side of some of the library's calls,
becomes the module ``lib/_native.so`` (the host compiler, torch's headers).
The library needs the CUDA toolchain alone: where the module cannot be built,
there is a warning and the library all the same, and only those calls raise.
Rebuilds only when a source or header is newer than the libraries, and the
module also when it was compiled for another Python or torch (``lib/_native.abi``).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "lib")
LIB_PATH = os.path.join(OUT_DIR, "libpaged_attn.so")
NATIVE_SRC = os.path.join(CSRC, "native_binding.cpp")
NATIVE_PATH = os.path.join(OUT_DIR, "_native.so")
NATIVE_ABI = os.path.join(OUT_DIR, "_native.abi")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return path


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = _sources()
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    files.append(os.path.abspath(__file__))
    return files


def _newer(target: str, files) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in files)


def up_to_date(lib_path: str = LIB_PATH) -> bool:
    return _newer(lib_path, _deps())


def native_abi() -> str:
    """What a compiled module depends on beside its sources: this Python, and this torch
    (its C++ classes, and where its libraries lie)."""
    import sysconfig

    import torch
    return "\n".join((sysconfig.get_config_var("SOABI") or sys.version, torch.__version__,
                      str(torch.version.git_version), str(torch._C._GLIBCXX_USE_CXX11_ABI),
                      os.path.dirname(torch.__file__)))


def native_fits() -> bool:
    """Whether the built module was compiled for this Python and this torch."""
    try:
        with open(NATIVE_ABI, encoding="utf-8") as f:
            return f.read() == native_abi()
    except OSError:
        return False


def native_up_to_date() -> bool:
    return _newer(NATIVE_PATH, [NATIVE_SRC, os.path.join(INCLUDE, "paged_attn.h"),
                                os.path.abspath(__file__)]) and native_fits()


def _compile_native() -> None:
    import sysconfig

    import torch
    where = os.path.dirname(torch.__file__)
    libs = os.path.join(where, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    includes = [INCLUDE, os.path.join(where, "include"),
                os.path.join(where, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], cuda]
    tmp = NATIVE_PATH + ".tmp"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{d}" for d in includes], NATIVE_SRC, "-o", tmp, f"-L{libs}", f"-Wl,-rpath,{libs}",
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the host compiler failed on {os.path.basename(NATIVE_SRC)}:\n{r.stdout}\n{r.stderr}")
    # (no stamp stands beside a module that it is not of)
    if os.path.exists(NATIVE_ABI):
        os.remove(NATIVE_ABI)
    os.replace(tmp, NATIVE_PATH)
    with open(NATIVE_ABI + ".tmp", "w", encoding="utf-8") as f:
        f.write(native_abi())
    os.replace(NATIVE_ABI + ".tmp", NATIVE_ABI)


def _try_native(running=None) -> None:
    """Builds the module, or waits for ``running``, which does; warns where that fails
    (and takes away a module of older sources)."""
    try:
        _compile_native() if running is None else running.result()
    except Exception as e:
        if os.path.exists(NATIVE_PATH):
            os.remove(NATIVE_PATH)
        warnings.warn(f"{os.path.basename(NATIVE_PATH)} was not built; the draft-tree and eviction "
                      f"calls of the Python binding will raise: {e}", RuntimeWarning, stacklevel=3)


def _native_done() -> bool:
    try:
        return native_up_to_date()
    except ImportError:  # without torch there is no module (the attempt will say so)
        return False


def _compile(src: str, obj: str, extra) -> None:
    cmd = [nvcc(), *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
           "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr", *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")


def build(force: bool = False, verbose: bool = False, extra=(), lib_path: str = LIB_PATH) -> str:
    """Compile and link the library; returns its path.

    ``extra`` adds nvcc flags (e.g. ``-DPKA_TIMELINE`` for the instrumented
    build); a build with extra flags goes to its own ``lib_path`` so that it
    never replaces the product library.
    """
    want_lib = force or not up_to_date(lib_path)
    want_native = lib_path == LIB_PATH and (force or not _native_done())
    if not want_lib and not want_native:
        return lib_path
    out_dir = os.path.dirname(lib_path)
    os.makedirs(out_dir, exist_ok=True)
    if not want_lib:
        _try_native()
        return lib_path
    srcs = _sources()
    objs = [os.path.join(out_dir, os.path.basename(s)[:-3] + ".o") for s in srcs]
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        futs = [ex.submit(_compile, s, o, list(extra)) for s, o in zip(srcs, objs)]
        native = ex.submit(_compile_native) if want_native else None
        for f in futs:
            f.result()
    tmp = lib_path + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    if native is not None:
        _try_native(native)
    if verbose:
        print(f"built {lib_path}", file=sys.stderr)
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
