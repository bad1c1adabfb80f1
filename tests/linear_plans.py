"""What flux_linear's plan takes for given sizes: tests/c_abi/linear_plans.cc,
compiled against the built library, asked on the CPU."""
import collections
import os
import subprocess
import tempfile

from diffusion_transformer_joint_gb300 import build

SINGLE, PAIR_W, PAIR_X = 0, 1, 2  # forms of linear_split
Plan = collections.namedtuple("Plan", "kernel form tile parts ns")
_HERE = os.path.dirname(os.path.abspath(__file__))
_ACT = {None: 0, "silu": 1, "gelu_tanh": 2, "swiglu": 3}


def plans(problems):
    """Plans of problems (B, S, K, N, kw) with kw's K2, act and residual."""
    lib = build.build()
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "linear_plans")
        libdir = os.path.dirname(lib)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", build.INCLUDE, "-I",
                        build.CSRC, "-I", os.path.join(cuda, "include"),
                        os.path.join(_HERE, "c_abi", "linear_plans.cc"), "-o", exe, "-L", libdir,
                        "-lflux_attn", "-L", os.path.join(cuda, "lib64"), "-lcudart",
                        f"-Wl,-rpath,{libdir}"], check=True, capture_output=True)
        lines = "".join(f"{B} {S} {K} {kw.get('K2', 0)} {N} {_ACT[kw.get('act')]} "
                        f"{int(kw.get('residual', False))}\n" for B, S, K, N, kw in problems)
        out = subprocess.run([exe], input=lines, check=True, capture_output=True, text=True).stdout
    got = []
    for line in out.splitlines():
        kernel, form, tile, parts, ns = line.split()
        got.append(Plan(kernel, int(form), int(tile), int(parts), float(ns)))
    assert len(got) == len(problems)
    return got
