"""What flux_linear's kernels leave behind when a bounded wait runs out. No GPU
fault is made: a copy of the library withholds one hand-off, so that the wait
ends by its clock, and the copy's kernel reports what it finds at its end."""
import ctypes
import shutil
import subprocess

import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R

pytestmark = pytest.mark.gpu

TIMEOUT = -7
NOT_LANDED, LEFT_EARLY = -77, -78  # reported by the copy's kernel, in place of the timeout

# What the copy of the split kernel withholds: the word that the call is given
# says it, and takes the kernel's report.
ALL_LATE, ONE_LATE, GIVES_UP, NO_ACCUMULATOR = 1, 2, 3, 4
WAIT = "if (!(ok = mbar_wait_cluster(bar_empty(s), (turn & 1u) ^ 1u, abort_flag))) break;"
REPORT = "if (tid == 0 && *abort_flag) atomicExch(status, FLUX_ERR_DEVICE_TIMEOUT);"
END = "cluster_wait();  // what this CTA sent has arrived: its shared memory may go"
SPLIT = ("linear_split_sm103a.cu", [
    ("const uint32_t sbase = smem_addr(base);",
     "const uint32_t sbase = smem_addr(base);\n"
     "  const int withheld = *status;\n  long long gave_up = 0;"),
    # stages are released from their second use on
    ("commit(bar_empty(s));",
     f"if (turn != 0 || !(withheld == {ALL_LATE} || (withheld == {ONE_LATE} && part == 0)))\n"
     "        commit(bar_empty(s));"),
    # a pair's even producer gives up at its second stage
    (WAIT, f"if (withheld == {GIVES_UP} && kPair && side == 0 && ks == k_lo + 1) {{\n"
           "        gave_up = clock64();\n        *abort_flag = 1;\n        ok = false;\n"
           "        break;\n      }\n      " + WAIT),
    ("commit(bar_acc);", f"if (withheld != {NO_ACCUMULATOR} || part != 0) commit(bar_acc);"),
    (END, "cluster_wait();\n  if (kC > 1 && !mbar_try_wait_cluster(bar_recv, 0)) "
          f"atomicMin(status, {NOT_LANDED});\n"),
    (REPORT, "if (gave_up != 0 && clock64() - gave_up < 2000000) "
             f"atomicMin(status, {LEFT_EARLY});\n"
             "  if (tid == 0 && *abort_flag) atomicMin(status, FLUX_ERR_DEVICE_TIMEOUT);"),
])
PAIR = ("linear_pair_sm103a.cu", [
    ("mma_commit_pair_elect(bar(kBarDrain), 0x1);",
     "if (cid != 0) mma_commit_pair_elect(bar(kBarDrain), 0x1);")])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _patched(path, name, patches):
    """flux_linear of a copy of the library with `patches` made in one source."""
    src = path / "csrc"
    shutil.copytree(build.CSRC, src)
    text = (src / name).read_text()
    for anchor, new in patches:
        assert text.count(anchor) == 1, f"not found exactly once: {anchor}"
        text = text.replace(anchor, new)
    (src / name).write_text(text)
    out = path / "libflux_patched.so"
    flags = [x for x in build.NVCC_FLAGS if x not in ("-Xptxas", "-v")]
    subprocess.run([build.nvcc(), *flags, "-I", build.INCLUDE, "-I", str(src),
                    *sorted(str(p) for p in src.glob("*.cu")), "-o", str(out)],
                   check=True, capture_output=True)
    lib = ctypes.CDLL(str(out))
    lib.flux_linear.argtypes = binding.load().flux_linear.argtypes
    lib.flux_linear.restype = ctypes.c_int
    return lib.flux_linear


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    return _patched(tmp_path_factory.mktemp("split"), *SPLIT)


@pytest.fixture(scope="module")
def pair(tmp_path_factory):
    return _patched(tmp_path_factory.mktemp("pair"), *PAIR)


def _problem(S, K, N):
    g = torch.Generator().manual_seed(71)
    x = torch.randn(1, S, K, generator=g).bfloat16().cuda()
    w = (torch.randn(N, K, generator=g) * K ** -0.5).bfloat16().cuda()
    return x, w, torch.randn(1, S, N, generator=g).bfloat16().cuda()


def _call(fn, x, w, residual, word=0):
    """The status word after a call that finds `word` there."""
    (_, S, K), N = x.shape, w.shape[0]
    out = torch.zeros(1, S, N, dtype=torch.bfloat16, device="cuda")
    status = torch.full((1,), word, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    rc = fn(x.data_ptr(), 0, K, K, None, 0, 0, 0, w.data_ptr(), K, 1, S, N, 0, None, None, 0, 0,
            residual.data_ptr(), 0, N, out.data_ptr(), 0, N, status.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    return int(status.item())


def _regular_still_works(x, w, residual):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.linear(x, w, residual=residual, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    R.check(got, R.linear(x, w, residual=residual), "after the timeout")


# Problems that run in the split kernel with the channels of a tile over two units
# or more: single CTAs, pairs over W's rows, pairs over token rows; the sums
# over the ring (first and last) and in a place of their own.
FORMS = [(9, 8192, 256), (100, 8192, 2048), (512, 8192, 256), (200, 8192, 4096)]


@pytest.mark.parametrize("late", [ONE_LATE, ALL_LATE])
@pytest.mark.parametrize("S,K,N", FORMS)
def test_sums_have_arrived_when_an_aborted_cluster_ends(split, S, K, N, late):
    """A unit that aborts, and one that waits for it, leave the cluster only
    after every unit's sums have landed in their shared memory."""
    x, w, res = _problem(S, K, N)
    assert _call(split, x, w, res, late) == TIMEOUT
    _regular_still_works(x, w, res)


@pytest.mark.parametrize("S,K,N", [(100, 1536, 2048), (512, 1536, 256)])
def test_a_pair_stays_for_copies_that_nobody_counts(split, S, K, N):
    """The even CTA's producer gives up at its second stage while the odd one
    goes on: no CTA leaves before the odd one's copies have had a millisecond."""
    x, w, res = _problem(S, K, N)
    assert _call(split, x, w, res, GIVES_UP) == TIMEOUT
    _regular_still_works(x, w, res)


@pytest.mark.parametrize("S,K,N", FORMS)
def test_the_wait_for_accumulators_reports(split, S, K, N):
    """The wait for a unit's accumulators, which an abort does not cut short, sets
    the status word when it runs out."""
    x, w, res = _problem(S, K, N)
    assert _call(split, x, w, res, NO_ACCUMULATOR) == TIMEOUT
    _regular_still_works(x, w, res)


def test_the_wait_for_the_last_mmas_reports(pair):
    x, w, res = _problem(2600, 64, 4096)
    assert _call(pair, x, w, res) == TIMEOUT
    _regular_still_works(x, w, res)
