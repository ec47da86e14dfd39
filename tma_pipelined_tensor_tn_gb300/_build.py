"""Build libtmagemm.so in-tree with nvcc for sm_103a (GB300).

Each ``csrc/*.cu`` is compiled to an object in parallel, then linked into a
shared library with the CUDA runtime linked statically, so the library loads
(and its symbols can be listed) on a machine without a GPU driver.  The binding
of the 8-bit operators (``csrc/torch_ops.cpp``, host code against torch's
headers) is compiled beside them into ``_torch_ops.so``, where torch is there to
compile it against; the library itself needs no torch.
"""
from __future__ import annotations

import glob
import hashlib
import os
import platform
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtmagemm.so")
# The checked build (-DTMAGEMM_CHECKED): kernels that check their own
# invariants and count the work units they complete.
BUILD_CHECKED = os.path.join(PKG, "_build_checked")
LIB_CHECKED = os.path.join(PKG, "libtmagemm_checked.so")

# The native binding of the 8-bit operators for torch tensors.
OPS = os.path.join(PKG, "_torch_ops.so")
OPS_SOURCE = os.path.join(CSRC, "torch_ops.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtmagemm.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _ops_command(out: str):
    """The compiler call for _torch_ops.so (this interpreter, this torch)."""
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
            "-I", sysconfig.get_paths()["include"], OPS_SOURCE, "-o", out,
            "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
            "-lc10_cuda", "-ltorch_cuda", "-ltorch"]


def _ops_stamp() -> str:
    import torch
    h = hashlib.sha256(" ".join((platform.machine(), sys.version, torch.__version__,
                                 " ".join(_ops_command(OPS)))).encode())
    for d in (OPS_SOURCE, os.path.join(INCLUDE, "tmagemm.h"), os.path.abspath(__file__)):
        with open(d, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def _start_ops(force: bool):
    """Starts compiling _torch_ops.so; None if it is up to date or there is no torch
    to compile it against."""
    try:
        import torch  # noqa: F401
    except (ImportError, OSError):
        return None
    if not force and os.path.exists(OPS) and os.path.exists(OPS + ".stamp"):
        with open(OPS + ".stamp") as f:
            if f.read().strip() == _ops_stamp():
                return None
    cmd = _ops_command(OPS + ".tmp")
    try:
        return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except OSError as e:     # no such compiler
        return cmd, str(e)


def _finish_ops(started) -> None:
    """Puts the compiled binding in place.  Where it does not compile, the library is
    still good for C callers: that is a warning, and no older binding is left behind,
    so that the 8-bit operators raise when they are called."""
    if started is None:
        return
    cmd, p = started
    out = p if isinstance(p, str) else p.communicate()[0].decode(errors="replace")
    if isinstance(p, str) or p.returncode != 0:
        for f in (OPS + ".stamp", OPS):
            if os.path.exists(f):
                os.remove(f)
        warnings.warn("compiling the torch binding failed:\n" + " ".join(cmd) + "\n" + out,
                      RuntimeWarning, stacklevel=3)
        return
    os.replace(OPS + ".tmp", OPS)
    with open(OPS + ".stamp", "w") as f:
        f.write(_ops_stamp() + "\n")


def _stamp(flags) -> str:
    """What a build depends on: this machine's architecture, the compiler
    flags and the bytes of every source and header."""
    h = hashlib.sha256()
    h.update(platform.machine().encode())
    h.update(" ".join(flags).encode())
    for d in sorted(_deps()):
        h.update(os.path.relpath(d, ROOT).encode())
        with open(d, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def up_to_date(lib: str = LIB, flags=None) -> bool:
    """True if `lib` exists and was built here from the current sources with
    these flags (a library built on another machine or from other sources is
    rebuilt)."""
    if flags is None:
        flags = ARCH + NVCC_FLAGS + (["-DTMAGEMM_CHECKED"] if lib == LIB_CHECKED else [])
    if not os.path.exists(lib) or not os.path.exists(lib + ".stamp"):
        return False
    with open(lib + ".stamp") as f:
        return f.read().strip() == _stamp(flags)


def build(force: bool = False, verbose: bool = False, extra_flags=None,
          checked: bool = False) -> str:
    """Compile every CUDA source and link libtmagemm.so (or, with checked=True,
    libtmagemm_checked.so), and the torch binding beside it where there is a torch;
    returns the library's path."""
    ops = _start_ops(force)
    try:
        return _build_library(force, verbose, extra_flags, checked)
    finally:
        _finish_ops(ops)


def _build_library(force: bool, verbose: bool, extra_flags, checked: bool) -> str:
    lib_path = LIB_CHECKED if checked else LIB
    build_dir = BUILD_CHECKED if checked else BUILD
    flags = ARCH + NVCC_FLAGS + (["-DTMAGEMM_CHECKED"] if checked else []) + list(extra_flags or [])
    if not force and up_to_date(lib_path, flags):
        return lib_path
    os.makedirs(build_dir, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in _sources():
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [cc, *flags, "-c", src, "-o", obj]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for cmd, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((cmd, text))
        elif verbose and text.strip():
            sys.stderr.write(text)
    if failed:
        msg = "\n".join(" ".join(c) + "\n" + t for c, t in failed)
        raise RuntimeError("nvcc failed:\n" + msg)
    tmp = lib_path + ".tmp"
    link = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + " ".join(link) + "\n" + r.stdout + r.stderr)
    os.replace(tmp, lib_path)
    with open(lib_path + ".stamp", "w") as f:
        f.write(_stamp(flags) + "\n")
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, checked="--checked" in sys.argv))
