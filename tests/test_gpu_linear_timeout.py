"""flux_linear's failure detection without a GPU fault: a hand-off is withheld
in a copy of the library, the kernel's bounded wait runs out, the status word
says so, and the regular library computes on the same context afterwards."""
import ctypes
import shutil
import subprocess
import time

import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R

pytestmark = pytest.mark.gpu

# the epilogue's release of its first accumulator (a pair's third tile waits for it)
PAIR = ("linear_pair_sm103a.cu",
        "if (lane == 0) mbar_arrive_cluster(acc_empty0 + 8u * static_cast<uint32_t>(lt & 1));",
        "if (lane == 0 && lt != 0) "
        "mbar_arrive_cluster(acc_empty0 + 8u * static_cast<uint32_t>(lt & 1));")
# the MMA warp's release of a stage (the producers wait to fill it again)
SPLIT = ("linear_split_sm103a.cu", "commit(bar_empty(s));",
         "if (turn != 0) commit(bar_empty(s));")


@pytest.mark.parametrize("patch,S,K,N,vecs", [(PAIR, 2600, 64, 4096, False),
                                              (PAIR, 2600, 64, 4096, True),
                                              (SPLIT, 9, 8192, 256, True),     # single CTAs
                                              (SPLIT, 100, 8192, 256, True)])  # CTA pairs
def test_bounded_wait_reports_timeout_and_context_survives(tmp_path, patch, S, K, N, vecs):
    build.build()
    binding.load()
    name, anchor, withheld = patch
    src = tmp_path / "csrc"
    shutil.copytree(build.CSRC, src)
    text = (src / name).read_text()
    assert text.count(anchor) == 1, "the hand-off to patch was not found exactly once"
    (src / name).write_text(text.replace(anchor, withheld))
    out = tmp_path / "libflux_withheld.so"
    flags = [x for x in build.NVCC_FLAGS if x not in ("-Xptxas", "-v")]
    subprocess.run([build.nvcc(), *flags, "-I", build.INCLUDE, "-I", str(src),
                    *sorted(str(p) for p in src.glob("*.cu")), "-o", str(out)],
                   check=True, capture_output=True)
    lib = ctypes.CDLL(str(out))
    lib.flux_linear.argtypes = binding.load().flux_linear.argtypes
    lib.flux_linear.restype = ctypes.c_int
    g = torch.Generator().manual_seed(61)
    x = torch.randn(1, S, K, generator=g).bfloat16().cuda()
    w = (torch.randn(N, K, generator=g) * K ** -0.5).bfloat16().cuda()
    y = torch.zeros(1, S, N, dtype=torch.bfloat16, device="cuda")
    bias = torch.randn(N, generator=g).bfloat16().cuda() if vecs else None
    gate = torch.randn(N, generator=g).bfloat16().cuda() if vecs else None
    P = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.time()
    rc = lib.flux_linear(x.data_ptr(), 0, K, K, None, 0, 0, 0, w.data_ptr(), K, 1, S, N, 0, P(bias),
                         P(gate), 0, 0, None, 0, 0, y.data_ptr(), 0, N, status.data_ptr(),
                         torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    elapsed = time.time() - t0
    assert int(status.item()) == -7, f"expected FLUX_ERR_DEVICE_TIMEOUT, got {int(status.item())}"
    assert elapsed < 60.0, f"bounded wait took {elapsed:.1f} s"
    status.zero_()
    got = binding.linear(x, w, bias=bias, gate=gate, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    rows = torch.tensor([0, S // 2, S - 1], device="cuda")
    R.check(got[:, rows], R.linear(x[:, rows], w, bias=bias, gate=gate), "after the timeout")
