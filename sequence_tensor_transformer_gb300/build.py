"""Builds libsptp.so in-tree from csrc/*.cu for sm_103a with nvcc.

Each translation unit is compiled in parallel to an object under _build/ and
the objects are linked into sequence_tensor_transformer_gb300/libsptp.so.  An
object is rebuilt when its source or any header is newer.

build(checked=True) builds the bounds-checked library libsptp_check.so
(objects under _build/check/): the same kernels compiled with
-DSPTP_BOUNDS_CHECK, which check every index and address they compute
against its buffer and report a failure as SPTP_ERR_BOUNDS in the workspace
status words.  It is a debug build for the tests, slower than the library.

csrc/decode_binding.cpp, a Python extension module over the installed torch's
headers, becomes _decode_binding.so beside the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsptp.so")
CHECKED_LIB = os.path.join(PKG, "libsptp_check.so")
BINDING = os.path.join(PKG, "_decode_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _build_binding() -> None:
    """The extension module for the torch and the Python that are in use: an
    object of its own for each of them, and a note of the object that the module
    was linked from, so that it is linked anew whenever that is another one.
    Where it cannot be compiled (no g++ or no Python.h) the library works
    without it, and a warning says so."""
    import torch

    home = os.path.dirname(os.path.abspath(torch.__file__))
    include = sysconfig.get_paths()["include"]
    src = os.path.join(CSRC, "decode_binding.cpp")
    where = hashlib.sha256(home.encode()).hexdigest()[:8]
    name = f"decode_binding-{torch.__version__}-{sysconfig.get_config_var('SOABI')}-{where}.o"
    obj, note = os.path.join(BUILD, name), os.path.join(BUILD, "decode_binding.linked")
    linked = None
    if os.path.exists(BINDING) and os.path.exists(note):
        with open(note) as f:
            linked = f.read()
    if shutil.which("g++") is None or not os.path.exists(os.path.join(include, "Python.h")):
        if linked != name and os.path.exists(BINDING):
            os.remove(BINDING)  # another torch's or Python's
        if not os.path.exists(BINDING):
            warnings.warn("no g++ or no Python.h: built without the extension module, a decoding step's calls cost "
                          "some microseconds more", RuntimeWarning)
        return
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    if _stale(obj, [src] + glob.glob(os.path.join(ROOT, "include", "*.h"))):
        dirs = [os.path.join(ROOT, "include"), os.path.join(home, "include"),
                os.path.join(home, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"), include]
        _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
             + ["-I" + d for d in dirs] + ["-c", src, "-o", obj + ".tmp"])
        os.replace(obj + ".tmp", obj)
    if linked != name or _stale(BINDING, [obj]):
        libs = ["torch_python", "torch", "torch_cpu", "c10", "c10_cuda"]
        _run(["g++", "-shared", "-o", BINDING + ".tmp", obj, "-L" + os.path.join(home, "lib")] + ["-l" + n for n in libs])
        if os.path.exists(note):
            os.remove(note)
        os.replace(BINDING + ".tmp", BINDING)
        with open(note, "w") as f:
            f.write(name)


def _run(cmd) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")


def build(verbose: bool = False, extra_flags=None, checked: bool = False) -> str:
    """Compile every CUDA source and link libsptp.so (checked: the
    bounds-checked libsptp_check.so); returns its path."""
    nvcc = _nvcc()
    objdir = os.path.join(BUILD, "check") if checked else BUILD
    lib_path = CHECKED_LIB if checked else LIB
    os.makedirs(objdir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdrs = _headers()
    flags = FLAGS + (["-DSPTP_BOUNDS_CHECK"] if checked else []) + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        if _stale(obj, [src] + hdrs) or extra_flags:
            cmd = [nvcc] + ARCH + flags + ["-c", src, "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(compile_one, srcs))
        binding.result()
    if _stale(lib_path, objs) or extra_flags:
        tmp = lib_path + ".tmp"
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    import sys
    print(build(verbose=True, checked="--checked" in sys.argv[1:]))
