"""Builds the CUDA library ``_lib/libfm.so`` in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel; the CUDA runtime is linked
statically, so the library needs only the driver (libcuda) at run time and
loads on a machine without a GPU (for the ABI checks).  ``build(debug=True)``
builds the same sources with the FM_DEBUG definition (device-side checks that
report FM_ERR_DEBUG_CHECK) into ``_lib/debug/libfm_debug.so``; the binding
loads it when the FM_LIBRARY environment variable names it.  Beside the library
stands ``_lib/_fm_call.so``, a CPython extension against the installed torch that
marshals the paged calls (host code only, whichever library is loaded), with a tag of the
torch and Python it fits.  The library does not need it: where it cannot be built
(no torch, no headers) build() warns, and the binding goes its slower way through ctypes.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libfm.so")
CALL = os.path.join(OUT_DIR, "_fm_call.so")
DEBUG_DIR = os.path.join(OUT_DIR, "debug")
DEBUG_LIB = os.path.join(DEBUG_DIR, "libfm_debug.so")
SOURCES = ["fm_api.cu", "fm_classify.cu", "fm_fwd.cu", "fm_bwd.cu", "fm_fp8.cu", "fm_compress.cu", "fm_noalloc.cu",
           "fm_paged.cu", "fm_paged_decode.cu", "fm_paged_chunk.cu", "fm_paged_weigh.cu", "fm_paged_evict.cu", "fm_rope.cu",
           "fm_verify.cu", "fm_mask.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfm.so")
    return p


def call_tag():
    """The torch and Python that an extension built now would fit; empty without torch."""
    try:
        import torch
    except ImportError:
        return ""
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"


def call_fits():
    """Whether the extension there was built against the installed torch and Python."""
    try:
        with open(CALL[:-2] + "tag") as f:
            return os.path.exists(CALL) and f.read() == call_tag() != ""
    except OSError:
        return False


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "fm.h"),
                                                                 os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files)


def _call_command(nvcc, out):
    """g++ command of the CPython extension (csrc/fm_call.cpp)."""
    import torch

    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-I{p}" for p in inc], os.path.join(CSRC, "fm_call.cpp"), "-o", out, f"-L{os.path.join(root, 'lib')}",
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _build_call(nvcc):
    """Compiles the extension and writes its tag."""
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = CALL + f".tmp{os.getpid()}"
    r = subprocess.run(_call_command(nvcc, tmp), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on fm_call.cpp:\n{r.stdout}\n{r.stderr}")
    with open(tmp + ".tag", "w") as f:
        f.write(call_tag())
    os.replace(tmp, CALL)
    os.replace(tmp + ".tag", CALL[:-2] + "tag")


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    lib = DEBUG_LIB if debug else LIB
    fresh = lambda f: not force and os.path.exists(f) and os.path.getmtime(f) >= _deps()  # noqa: E731
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        call = None if fresh(CALL) and call_fits() else ex.submit(lambda: _build_call(_nvcc()))
        if not fresh(lib):
            _build_lib(lib, verbose, debug)
        try:
            if call is not None:
                call.result()
        except (ImportError, OSError, RuntimeError) as e:
            warnings.warn(f"the paged calls go through ctypes, about 10 us more each: {e}", RuntimeWarning, stacklevel=2)
    return lib


def _build_lib(lib, verbose, debug):
    out_dir = os.path.dirname(lib)
    os.makedirs(out_dir, exist_ok=True)
    nvcc = _nvcc()
    common = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-I", INCLUDE, "-I", CSRC, *ARCH]
    if debug:
        common += ["-DFM_DEBUG"]
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(out_dir, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *common, "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cpp"):
            cmd = [nvcc, "-x", "c++", *common, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, err in results:
            if err:
                print(err)
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *[o for o, _ in results],
           "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv))
