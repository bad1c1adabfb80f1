"""flux_linear_fp8's split kernel: every tile with every number of parts
(tests/split_parts_cases.py)."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R
from tests import fp8_reference as F
from tests import operator_plans as P
from tests import split_parts_cases as C

_ALL = [(key, act) for act, cases in ((None, C.LINEAR), ("swiglu", C.GLU)) for key in cases]


def test_the_cases_take_their_tiles_and_parts():
    lines = [P.linear(1, *(C.GLU if act else C.LINEAR)[key], act=act, residual=True)
             for key, act in _ALL]
    assert [p[:3] for p in P.plans(lines)] == [("split", *key) for key, _ in _ALL]
    parts = {1, 2, 3, 4, 5, 6, 8}
    for cases in (C.LINEAR, C.GLU):
        # (128 tokens and all channels: hardly ever the estimate's pick)
        assert set(cases) == {(q, c) for q in (16, 32, 64, 96, 128) for c in parts} - {(128, 1)}


@pytest.mark.gpu
@pytest.mark.parametrize("key,act", _ALL)
def test_every_row_and_feature(key, act):
    """All of the output against 64 bits, rows around it left as they were, and the
    same bits from a graph."""
    build.build()
    S, K, N = (C.GLU if act else C.LINEAR)[key]
    g = torch.Generator().manual_seed(S + K + N)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rows = 2 * N if act else N
    x, xs = binding.quantize_fp8((r(S, K) * torch.exp(r(S, 1))).bfloat16().cuda())
    w, ws = binding.quantize_fp8((r(rows, K) * K ** -0.5).bfloat16().cuda(), rows=128)
    ops = dict(bias=r(rows).cuda(), gate=r(N).cuda(), residual=r(S, N).bfloat16().cuda())
    around = torch.full((S + 2, N + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    out = around[1:-1, :N]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        binding.linear_fp8(x, xs, w, ws, act=act, out=out, status=status, **ops)

    call()
    torch.cuda.synchronize()
    first = out.clone()
    assert int(status.item()) == 0
    R.check(first, F.linear(x, xs, w, ws, act=act, **ops), f"{key} {act}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(out.contiguous().view(torch.int16), first.view(torch.int16))
    assert bool((around[0] == 5).all() and (around[-1] == 5).all() and (around[:, N:] == 5).all())
