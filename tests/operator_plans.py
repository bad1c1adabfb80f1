"""What the plans of flux_linear_fp8 and flux_cross_attention take for given
sizes: tests/c_abi/operator_plans.cc, compiled against the built library, asked on
the CPU."""
import os
import subprocess
import tempfile

from diffusion_transformer_joint_gb300 import build

_HERE = os.path.dirname(os.path.abspath(__file__))
_ACT = {None: 0, "silu": 1, "gelu_tanh": 2, "swiglu": 3}


def linear(B, S, K, N, act=None, residual=False, **_):
    return f"linear {B} {S} {K} {N} {_ACT[act]} {int(residual)}\n"


def cross(B, Sq, Sk, H, Hk, D):
    return f"cross {B} {Sq} {Sk} {H} {Hk} {D}\n"


def plans(lines):
    """(form, tile or parts, parts, ns) for each line made by linear() or cross()."""
    lib = build.build()
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "operator_plans")
        libdir = os.path.dirname(lib)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", build.INCLUDE, "-I",
                        build.CSRC, "-I", os.path.join(cuda, "include"),
                        os.path.join(_HERE, "c_abi", "operator_plans.cc"), "-o", exe, "-L", libdir,
                        "-lflux_attn", "-L", os.path.join(cuda, "lib64"), "-lcudart",
                        f"-Wl,-rpath,{libdir}"], check=True, capture_output=True)
        out = subprocess.run([exe], input="".join(lines), check=True, capture_output=True,
                             text=True).stdout
    got = [line.split() for line in out.splitlines()]
    assert len(got) == len(lines)
    return [(f, int(a), int(b), float(ns)) for f, a, b, ns in got]
