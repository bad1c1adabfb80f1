"""Every kernel, form and tile of flux_linear_fp8's and flux_cross_attention's
plans (tests/operator_cases.py), eagerly and replayed from a graph."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R
from tests import cross_reference as X
from tests import fp8_reference as F
from tests import operator_cases as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _twice(fn, out):
    """fn() once, then replayed from a graph over other contents of `out`."""
    fn()
    torch.cuda.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    out.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("key,act", [(k, None) for k in C.LINEAR] + [(k, "swiglu") for k in C.GLU])
def test_linear_fp8(key, act):
    B, S, K, N, kw = (C.GLU if act else C.LINEAR)[key]
    kw = dict(kw)
    act = kw.pop("act", act)
    g = torch.Generator().manual_seed(S + K)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rows = 2 * N if act == "swiglu" else N
    x, xs = binding.quantize_fp8((r(B, S, K) * torch.exp(r(B, S, 1))).bfloat16().cuda())
    w, ws = binding.quantize_fp8((r(rows, K) * K ** -0.5).bfloat16().cuda(), rows=128)
    ops = dict(bias=r(rows).cuda() if kw.get("bias") else None,
               gate=r(B, N).cuda() if kw.get("gate") else None,
               residual=r(B, S, N).bfloat16().cuda() if kw.get("residual") else None)
    out = torch.empty(B, S, N, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _twice(lambda: binding.linear_fp8(x, xs, w, ws, act=act, out=out, status=status, **ops), out)
    assert int(status.item()) == 0
    # some rows and all features, and some features of all rows
    at = torch.tensor(sorted({0, S // 3, S - 1}), device="cuda")
    part = dict(ops, residual=None if ops["residual"] is None else ops["residual"][:, at])
    R.check(out[:, at], F.linear(x[:, at], xs[:, at], w, ws, act=act, **part), "rows")
    if act is None or act == "silu":
        lo = N - N % 128 - 128 if N % 128 else N - 128
        cols = dict(bias=None if ops["bias"] is None else ops["bias"][lo:],
                    gate=None if ops["gate"] is None else ops["gate"][:, lo:],
                    residual=None if ops["residual"] is None else ops["residual"][..., lo:])
        R.check(out[..., lo:], F.linear(x, xs, w[lo:], ws[lo // 128:], act=act, **cols), "features")


@pytest.mark.parametrize("keys", ["all", "lengths", "mask"])
@pytest.mark.parametrize("key", list(C.CROSS))
def test_cross_attention(key, keys):
    B, Sq, Sk, H, Hk, D = C.CROSS[key]
    g = torch.Generator().manual_seed(Sq + Sk)
    q, k, v = (torch.randn(B, n, h, D, generator=g).bfloat16().cuda()
               for n, h in ((Sq, H), (Sk, Hk), (Sk, Hk)))
    kw = {}
    if keys == "lengths":
        kw["lengths"] = torch.tensor([Sk - 3, Sk // 2 + 1][:B], dtype=torch.int32, device="cuda")
    if keys == "mask":
        kw["mask"] = (torch.rand(B, Sk, generator=g) < 0.8).cuda()
    out = torch.empty_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _twice(lambda: binding.cross_attention(q, k, v, out=out, status=status, **kw), out)
    assert int(status.item()) == 0
    at = torch.tensor(sorted({0, 1 % Sq, Sq // 3, Sq // 2, Sq - 1}), device="cuda")
    R.check(out[:, at], X.cross(q[:, at], k, v, **kw), f"{key} {keys}")
