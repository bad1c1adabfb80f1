"""The library's own status word: calls that are given none report to it, eager
or captured, and take_status reads and clears it."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _python(code, **env):
    """Runs `code` in a process of its own."""
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=dict(os.environ, **env),
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr


def test_null_and_no_device():
    build.build()
    lib = binding.load()
    assert lib.flux_status_word(None) == -1
    if not torch.cuda.is_available():
        assert lib.flux_take_status(None) in (-6, -8)


@pytest.mark.gpu
def test_a_call_without_status_allocates_nothing_but_its_output():
    build.build()
    x = torch.randn(1, 5, 64, device="cuda").bfloat16()
    w = torch.randn(128, 64, device="cuda").bfloat16()
    out = binding.linear(x, w)
    torch.cuda.synchronize()
    n = torch.cuda.memory_stats()["allocation.all.allocated"]
    binding.linear(x, w, out=out)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == n
    assert binding.take_status() == 0


FIRST_CALL_CAPTURED = """
import torch
from diffusion_transformer_joint_gb300 import binding
x = torch.randn(1, 9, 64, device="cuda").bfloat16()
w = torch.randn(128, 64, device="cuda").bfloat16()
wp = torch.randn(3 * 128 + 256, 64, device="cuda").bfloat16()
out = torch.zeros(1, 9, 128, device="cuda").bfloat16()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    binding.linear(x, w, out=out)
    q, k, v, act = binding.qkv_mlp_proj(x, wp, 1, 128)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, binding.linear(x, w))
assert all(torch.equal(a, b) for a, b in zip((q, k, v, act), binding.qkv_mlp_proj(x, wp, 1, 128)))
assert binding.take_status() == 0
"""


@pytest.mark.gpu
def test_the_first_call_may_be_a_captured_one():
    build.build()
    _python(FIRST_CALL_CAPTURED)


TIMEOUT_SEEN = """
import torch
from diffusion_transformer_joint_gb300 import binding
x = torch.randn(1, 9, 8192, device="cuda").bfloat16()
w = torch.randn(256, 8192, device="cuda").bfloat16()
assert binding.take_status() == 0
binding.linear(x, w)
binding.modulated_norm(x)
assert binding.take_status() == -7
assert binding.take_status() == 0
own = torch.zeros(1, dtype=torch.int32, device="cuda")
binding.linear(x, w, status=own)
torch.cuda.synchronize()
assert int(own.item()) == -7 and binding.take_status() == 0
"""


@pytest.mark.gpu
def test_a_timeout_of_a_call_without_status_is_seen(tmp_path):
    """A hand-off is withheld in a copy of the library (as in the tests of the
    bounded waits); the binding loads the copy."""
    src = tmp_path / "csrc"
    shutil.copytree(build.CSRC, src)
    f = src / "linear_split_sm103a.cu"
    text = f.read_text()
    assert text.count("commit(bar_empty(s));") == 1
    f.write_text(text.replace("commit(bar_empty(s));", "if (turn != 0) commit(bar_empty(s));"))
    out = tmp_path / "libflux_withheld.so"
    flags = [x for x in build.NVCC_FLAGS if x not in ("-Xptxas", "-v")]
    subprocess.run([build.nvcc(), *flags, "-I", build.INCLUDE, "-I", str(src),
                    *sorted(str(p) for p in src.glob("*.cu")), "-o", str(out)],
                   check=True, capture_output=True)
    _python(TIMEOUT_SEEN, FLUX_ATTN_LIB=str(out))
