"""flux_linear behind a kernel of another library that lets its dependents start
at once and then runs for longer than the budget of a bounded wait: the product
waits for it without counting that time as its own."""
import ctypes
import subprocess

import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R

pytestmark = pytest.mark.gpu

# One block: triggers, spins for `cycles` (the budget is 2e9), then copies n words.
SOURCE = r"""
#include <cuda_runtime.h>
__global__ void long_kernel(const int *src, int *dst, int n, long long cycles) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long t0 = clock64();
  while (clock64() - t0 < cycles) {
  }
  for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}
extern "C" int run(const void *src, void *dst, int n, long long cycles, void *stream) {
  long_kernel<<<1, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const int *>(src), static_cast<int *>(dst), n, cycles);
  return static_cast<int>(cudaGetLastError());
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    build.build()
    binding.load()
    d = tmp_path_factory.mktemp("long_kernel")
    (d / "long_kernel.cu").write_text(SOURCE)
    flags = [x for x in build.NVCC_FLAGS if x not in ("-Xptxas", "-v")]
    subprocess.run([build.nvcc(), *flags, str(d / "long_kernel.cu"), "-o", str(d / "long.so")],
                   check=True, capture_output=True)
    fn = ctypes.CDLL(str(d / "long.so")).run
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong,
                   ctypes.c_void_p]
    return fn


@pytest.mark.parametrize("S,K,N", [(2600, 64, 4096),   # linear_pair
                                   (9, 8192, 256)])    # linear_split
def test_time_of_the_kernel_before_is_not_counted(run, S, K, N):
    g = torch.Generator().manual_seed(81)
    src = torch.randn(1, S, K, generator=g).bfloat16().cuda()
    w = (torch.randn(N, K, generator=g) * K ** -0.5).bfloat16().cuda()
    x = torch.zeros_like(src)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(1, S, N, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    assert run(src.data_ptr(), x.data_ptr(), src.numel() // 2, 2_600_000_000,
               torch.cuda.current_stream().cuda_stream) == 0
    binding.linear(x, w, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    rows = torch.tensor([0, S // 2, S - 1], device="cuda")
    R.check(out[:, rows], R.linear(src[:, rows], w), "behind a long kernel")
