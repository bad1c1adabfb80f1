"""The scale of flux_cross_attention and binding.cross_attention: whatever the
kernel cannot take as it is given is refused, neither replaced nor overflowed."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests.test_fp8_cross_host import _call, _on_device

TOP = 2.0 ** 127
LEAST = 2.0 ** -149  # the smallest fp32 above zero


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses stay off a GPU")
@pytest.mark.parametrize("scale", [0.0, LEAST, 1.0, TOP])
def test_accepts(lib, scale):
    assert _on_device(_call(lib, "flux_cross_attention", dict(scale=scale)))


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses stay off a GPU")
@pytest.mark.parametrize("scale", [TOP * (1 + 2.0 ** -23), 3e38])
def test_refuses_what_log2e_takes_past_fp32(lib, scale):
    """Scores times scale log2(e): an infinite factor makes NaN of a score of 0."""
    assert _call(lib, "flux_cross_attention", dict(scale=scale)) == -2


@pytest.mark.parametrize("scale", [0.0, -1.0, 1e-50, LEAST / 2, TOP * 1.001, 2.9e38, 1e300,
                                   float("nan"), float("inf")])
def test_binding_refuses(scale):
    """1e-50 is 0 in fp32, which would stand for 1 / sqrt(D)."""
    with pytest.raises(ValueError, match="scale"):
        binding._softmax_scale(scale)


def test_binding_accepts():
    assert binding._softmax_scale(None) == 0.0
    for scale in (LEAST, 0.25, 1, TOP):
        assert binding._softmax_scale(scale) == scale


@pytest.mark.gpu
@pytest.mark.parametrize("stream", [False, True])  # compiled marshalling, and Python's
def test_calls(lib, stream):
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(2, n, 4, 64, generator=g).bfloat16().cuda() for n in (5, 40, 40))
    kw = dict(stream=torch.cuda.current_stream()) if stream else {}
    for scale in (1e-50, 2.9e38, 0.0):
        with pytest.raises(ValueError, match="scale"):
            binding.cross_attention(q, k, v, scale=scale, **kw)
    # the least scale: all weights are the same
    got = binding.cross_attention(q, k, v, scale=LEAST, **kw).double()
    want = v.double().mean(1, keepdim=True).expand_as(got)
    # (p = 1 and sums of 40 in fp32, one rounding to bf16)
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -17 * v.double().abs().mean(1, keepdim=True)
    assert bool(((got - want).abs() <= bound).all())
    # the largest, over scores of 0 (an infinite factor would make NaN of them)
    got = binding.cross_attention(torch.zeros_like(q), k, v, scale=TOP, **kw).double()
    assert bool(((got - want).abs() <= bound).all())
    assert binding.take_status() == 0
