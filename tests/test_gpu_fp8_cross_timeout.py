"""Failure detection of the 8-bit products and the cross-attention without a GPU
fault: hand-offs are withheld in a copy of the library, the kernels' bounded waits
run out, the status word says so, and the regular library computes on the same
context afterwards."""
import ctypes
import shutil
import subprocess
import time

import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R
from tests import cross_reference as X
from tests import fp8_reference as F

pytestmark = pytest.mark.gpu

PATCHES = (
    # the sums' release of an accumulator (the MMAs of a later group wait for it)
    ("linear_fp8_pair_sm103a.cu",
     "if (lane == 0) mbar_arrive_cluster_relaxed(acc_empty0 + 8u * a);",
     "if (lane == 0 && n != 0) mbar_arrive_cluster_relaxed(acc_empty0 + 8u * a);"),
    # the MMA warp's release of a stage (the producer waits to fill it again)
    ("linear_fp8_split_sm103a.cu", "mma_commit_elect(bar(T::kEmpty + s));",
     "if (turn != 0) mma_commit_elect(bar(T::kEmpty + s));"),
    # the softmax's hand-over of P
    ("cross_attention_sm103a.cu",
     "tc_fence_before_sync();\n        warp_arrive(bar(L::kPFull + t), lane);\n      }",
     "tc_fence_before_sync();\n        if (g != 1) warp_arrive(bar(L::kPFull + t), lane);\n      }"),
)


@pytest.fixture(scope="module")
def withheld(tmp_path_factory):
    build.build()
    regular = binding.load()
    tmp = tmp_path_factory.mktemp("withheld")
    src = tmp / "csrc"
    shutil.copytree(build.CSRC, src)
    for name, anchor, instead in PATCHES:
        text = (src / name).read_text()
        assert text.count(anchor) == 1, f"the hand-off to patch was not found exactly once: {name}"
        (src / name).write_text(text.replace(anchor, instead))
    out = tmp / "libflux_withheld.so"
    flags = [x for x in build.NVCC_FLAGS if x not in ("-Xptxas", "-v")]
    subprocess.run([build.nvcc(), *flags, "-I", build.INCLUDE, "-I", str(src),
                    *sorted(str(p) for p in src.glob("*.cu")), "-o", str(out)],
                   check=True, capture_output=True)
    lib = ctypes.CDLL(str(out))
    for name in ("flux_linear_fp8", "flux_cross_attention"):
        getattr(lib, name).argtypes = getattr(regular, name).argtypes
        getattr(lib, name).restype = ctypes.c_int
    return lib


class _With:
    """The binding over another library for one call."""

    def __init__(self, lib, name):
        regular = binding.load()

        class Proxy:
            def __getattr__(self, n):
                return getattr(lib if n == name else regular, n)

        self.lib, self.regular = Proxy(), regular

    def __enter__(self):
        binding._lib = self.lib

    def __exit__(self, *_):
        binding._lib = self.regular


def _check(lib, name, call, want, rows):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.time()
    with _With(lib, name):
        call(status)
    torch.cuda.synchronize()
    assert time.time() - t0 < 60.0
    assert int(status.item()) == -7, f"expected FLUX_ERR_DEVICE_TIMEOUT, got {int(status.item())}"
    status.zero_()
    got = call(status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    R.check(got[:, rows], want, "after the timeout")


@pytest.mark.parametrize("S,K,N", [(2600, 1024, 4096), (700, 4096, 1024),  # CTA pairs
                                   (9, 8192, 256), (120, 8192, 4096)])     # clusters of single CTAs
@pytest.mark.parametrize("residual", [False, True])
def test_linear_fp8(withheld, S, K, N, residual):
    g = torch.Generator().manual_seed(61)
    x, xs = binding.quantize_fp8(torch.randn(1, S, K, generator=g).cuda())
    w, ws = binding.quantize_fp8((torch.randn(N, K, generator=g) * K ** -0.5).cuda(), rows=128)
    bias = torch.randn(N, generator=g).cuda()
    res = torch.randn(1, S, N, generator=g).bfloat16().cuda() if residual else None
    rows = torch.tensor([0, S // 2, S - 1], device="cuda")
    want = F.linear(x[:, rows], xs[:, rows], w, ws, bias=bias,
                    residual=None if res is None else res[:, rows])
    _check(withheld, "flux_linear_fp8",
           lambda status: binding.linear_fp8(x, xs, w, ws, bias=bias, residual=res, status=status),
           want, rows)


@pytest.mark.parametrize("B,Sq,Sk,H", [(2, 700, 600, 4), (1, 5, 3000, 8), (2, 40, 700, 32)])
@pytest.mark.parametrize("lengths", [False, True])
def test_cross_attention(withheld, B, Sq, Sk, H, lengths):
    g = torch.Generator().manual_seed(71)
    q, k, v = (torch.randn(B, n, H, 128, generator=g).bfloat16().cuda() for n in (Sq, Sk, Sk))
    kw = dict(lengths=torch.full((B,), Sk - 5, dtype=torch.int32, device="cuda")) if lengths else {}
    rows = torch.tensor([0, Sq - 1], device="cuda")
    _check(withheld, "flux_cross_attention",
           lambda status: binding.cross_attention(q, k, v, status=status, **kw),
           X.cross(q[:, rows], k, v, **kw), rows)


@pytest.fixture(scope="module")
def impatient(tmp_path_factory):
    """A copy of the library whose waits are given 150 000 cycles (75 us)."""
    regular = binding.load()
    tmp = tmp_path_factory.mktemp("impatient")
    src = tmp / "csrc"
    shutil.copytree(build.CSRC, src)
    text = (src / "ptx_sm103a.cuh").read_text()
    assert text.count("kWaitBudgetCycles = 2000000000LL") == 1
    (src / "ptx_sm103a.cuh").write_text(
        text.replace("kWaitBudgetCycles = 2000000000LL", "kWaitBudgetCycles = 150000LL"))
    out = tmp / "libflux_impatient.so"
    flags = [x for x in build.NVCC_FLAGS if x not in ("-Xptxas", "-v")]
    subprocess.run([build.nvcc(), *flags, "-I", build.INCLUDE, "-I", str(src),
                    *sorted(str(p) for p in src.glob("*.cu")), "-o", str(out)],
                   check=True, capture_output=True)
    lib = ctypes.CDLL(str(out))
    lib.flux_cross_attention.argtypes = regular.flux_cross_attention.argtypes
    lib.flux_cross_attention.restype = ctypes.c_int
    return lib


@pytest.mark.parametrize("B,Sq,Sk,lengths", [
    (1, 256, 131072, None),           # an item of a millisecond
    (2, 38912, 32768, (32768, 300)),  # tiles with left-out keys after many items without
    (1, 2, 524288, None),             # a cluster's parts
    (1, 2, 524288, (524200,))])
def test_long_items_are_no_timeout(impatient, B, Sq, Sk, lengths):
    g = torch.Generator().manual_seed(81)
    q, k, v = (torch.randn(B, n, 1, 128, generator=g).bfloat16().cuda() for n in (Sq, Sk, Sk))
    kw = {} if lengths is None else dict(lengths=torch.tensor(lengths, dtype=torch.int32).cuda())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with _With(impatient, "flux_cross_attention"):
        got = binding.cross_attention(q, k, v, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    rows = torch.tensor([0, Sq - 1], device="cuda")
    R.check(got[:, rows], X.cross(q[:, rows], k, v, **kw), "long")
