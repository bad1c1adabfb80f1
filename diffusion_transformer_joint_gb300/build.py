"""Builds the CUDA library libflux_attn.so in-tree with nvcc for sm_103a.

Usage: ``python -m diffusion_transformer_joint_gb300.build [--force] [--checked]``.
The binding's compiled marshalling is built beside it (marshal.cpp, with g++ and
torch's headers) where those are there; without it calls are marshalled in Python.
``--checked`` builds libflux_attn_checked.so instead: the same library compiled
with -DFLUX_DEBUG, whose attention kernel checks its shared-memory, TMEM, TMA
and exchange-buffer accesses and reports a failed check in the status word
(the binding loads it when FLUX_ATTN_DEBUG=1).
"""
from __future__ import annotations

import glob
import hashlib
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libflux_attn.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
CHECKED_LIB_PATH = os.path.join(BUILD_DIR, "libflux_attn_checked.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17", "--threads", "0",
    "-Xcompiler", "-fPIC,-O2", "-shared",
    "-Xptxas", "-v",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(
        glob.glob(os.path.join(CSRC, "*.h"))) + sorted(glob.glob(os.path.join(INCLUDE, "*.h")))


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def marshal_path() -> str:
    """Where the compiled marshalling lies, built for this torch and this Python from
    these sources: a changed prototype asks for another file, never an older one's
    calls."""
    import torch

    digest = hashlib.sha256()
    for p in _marshal_inputs():
        with open(p, "rb") as f:
            digest.update(f.read())
    return os.path.join(BUILD_DIR, f"torch-{torch.__version__}",
                        f"_marshal-{digest.hexdigest()[:16]}"
                        + sysconfig.get_config_var("EXT_SUFFIX"))


def _marshal_inputs():
    return [os.path.join(PKG, "marshal.cpp"), os.path.join(INCLUDE, "flux_attn.h")]


def build_marshal(force: bool = False) -> str:
    """Compile marshal.cpp against this torch; returns its path."""
    import torch

    src, out = _marshal_inputs()[0], marshal_path()
    if not force and os.path.exists(out):
        return out
    os.makedirs(os.path.dirname(out), exist_ok=True)
    top = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = out + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-isystem", os.path.join(top, "include"),
           "-isystem", os.path.join(top, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(cuda, "include"), "-I", INCLUDE, src, "-o", tmp,
           "-L", os.path.join(top, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", f"-Wl,-rpath,{os.path.join(top, 'lib')}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed on marshal.cpp")
    os.replace(tmp, out)
    return out


def build(force: bool = False, out: str = LIB_PATH, defines=(), verbose: bool = False) -> str:
    """Compile every csrc/*.cu into one shared library; returns its path."""
    os.makedirs(os.path.dirname(out), exist_ok=True)
    if not force and os.path.exists(out):
        t = os.path.getmtime(out)
        if all(os.path.getmtime(p) <= t for p in _inputs()):
            return out
    tmp = out + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC,
           *[f"-D{d}" for d in defines], *sources(), "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    log = os.path.join(os.path.dirname(out), "nvcc.log")
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + res.stdout + res.stderr)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"nvcc failed (log: {log})")
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(tmp, out)
    return out


def build_checked(force: bool = False, out: str = CHECKED_LIB_PATH) -> str:
    """The checked library (-DFLUX_DEBUG) at ``out``; returns its path."""
    return build(force=force, out=out, defines=("FLUX_DEBUG",))


def try_build_marshal(force: bool = False):
    """build_marshal(), or None and a message where g++ or torch's headers are missing:
    the binding then marshals every call in Python."""
    try:
        return build_marshal(force)
    except (ImportError, OSError, RuntimeError) as e:
        sys.stderr.write(f"compiled marshalling not built ({e}): calls are marshalled in Python\n")
        return None


def main() -> int:
    if "--checked" in sys.argv:
        print(build_checked(force="--force" in sys.argv))
        return 0
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    path = try_build_marshal(force="--force" in sys.argv)
    if path is not None:
        print(path)
    return 0


if __name__ == "__main__":
    sys.exit(main())
