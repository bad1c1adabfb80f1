"""Sizes that the C ABI takes as an int: 2^32 + 64 channels are refused, not
taken for 64. (Memory is reserved, not touched: the calls are refused first.)"""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build

pytestmark = pytest.mark.gpu

FAR = 2 ** 32 + 64


@pytest.fixture(autouse=True)
def _lib():
    build.build()
    binding.load()
    yield
    torch.cuda.empty_cache()


def test_norm_refuses_channels_past_an_int():
    x = torch.empty(1, FAR, dtype=torch.bfloat16, device="cuda")
    with pytest.raises((ValueError, binding.FluxError)):
        binding.modulated_norm(x, out=torch.empty_like(x))


def test_linear_refuses_channels_past_an_int():
    x = torch.empty(1, FAR, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(8, FAR, dtype=torch.bfloat16, device="cuda")
    with pytest.raises((ValueError, binding.FluxError)):
        binding.linear(x, w)
    x2 = torch.empty(1, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(8, FAR + 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises((ValueError, binding.FluxError)):
        binding.linear(x2, w, x2=x)


def test_refuses_batches_past_an_int():
    x = torch.empty(2 ** 32 + 1, 1, 8, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(x)
    with pytest.raises((ValueError, binding.FluxError)):
        binding.modulated_norm(x, out=out)
    with pytest.raises((ValueError, binding.FluxError)):
        binding.linear(x, torch.empty(8, 8, dtype=torch.bfloat16, device="cuda"), out=out)
