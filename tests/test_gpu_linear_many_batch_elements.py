"""binding.linear over few tokens each of many batch elements that do not follow
one another in memory."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


@pytest.mark.parametrize("B,S", [(20, 3), (31, 2), (32, 2), (100, 2), (9, 7), (8, 8)])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_views_of_few_tokens(B, S, act):
    K, N = 264, 200
    g = torch.Generator().manual_seed(B)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()  # noqa: E731
    rows = 2 * N if act == "swiglu" else N
    ops = dict(x=r(B, S + 3, K)[:, 2:-1], w=r(rows, K) / 16, bias=r(rows), gate=r(B, N), act=act,
               residual=r(B, S + 1, N)[:, 1:])
    buf = torch.full((B, S + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.linear(**ops, out=buf[:, 1:-1], status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    R.check(out, R.linear(**ops), f"{B}x{S}")
    assert bool((buf[:, 0] == 7).all() and (buf[:, -1] == 7).all())
