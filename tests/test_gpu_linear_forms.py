"""binding.linear in every kernel, form, split and tile width of its plan, against
the 64-bit definition, and at the sizes of the FLUX.2 blocks."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R
from tests import linear_cases as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _make(B, S, K, N, K2=0, act=None, bias=False, gate=False, residual=False, vec=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(B + S + K + N)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows = 2 * N if act == "swiglu" else N
    ops = dict(x=r(B, S, K).bfloat16(), w=(r(rows, K + K2) * (K + K2) ** -0.5).bfloat16(), act=act)
    if K2:
        ops["x2"] = r(B, S, K2).bfloat16()
    if bias:
        ops["bias"] = r(rows).to(vec)
    if gate:
        ops["gate"] = r(B, N).to(vec)
    if residual:
        ops["residual"] = (2 * r(B, S, N)).bfloat16()
    return ops


def _run(ops, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.linear(status=status, **ops, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out


@pytest.mark.parametrize("case", [c for _, c in C.CLASSES], ids=lambda c: "x".join(
    str(n) for n in c[:3]) + ("-swiglu" if c[3].get("act") == "swiglu" else ""))
def test_every_class(case):
    S, K, N, kw = case
    ops = _make(1, S, K, N, **kw, bias=True, gate=True, residual=True,
                vec=(torch.bfloat16, torch.float32)[S % 2])
    ref = R.linear(**ops)
    R.check(_run(ops), ref, "apart")
    R.check(_run(ops, out=ops["residual"]), ref, "in place")


@pytest.mark.parametrize("case", [c for _, c in C.WIDE_VIEWS])
def test_wide_tiles_over_views(case):
    """Trailing tokens and a column range of wider buffers, updated in place; what
    lies around them is left as it was."""
    B, S, K, N, kw = case
    ops = _make(B, S, K, N, **kw, bias=True, gate=True, residual=True, vec=torch.float32)
    for name in ("x", "x2"):
        if name in ops:
            t = ops[name]
            buf = torch.full((B, S + 3, t.shape[2] + 8), float("nan"), dtype=t.dtype, device="cuda")
            buf[:, 3:, 8:] = t
            ops[name] = buf[:, 3:, 8:]
    buf = torch.full((B, S + 5, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    stream = buf[:, 4:-1, 8:-16]
    stream.copy_(ops["residual"])
    ref = R.linear(**ops)
    assert _run(dict(ops, residual=stream), out=stream) is stream
    R.check(stream, ref, "views")
    stream.fill_(7.0)
    assert bool((buf == 7.0).all())


@pytest.mark.parametrize("name", list(C.WORKLOADS))
def test_block_sizes(name):
    """Rows from both ends and both sides of every border of 32, 64 and 128 rows,
    and drawn ones, over all features."""
    B, S, K, N, kw = C.WORKLOADS[name]
    ops = _make(B, S, K, N, **kw)
    out = _run(ops)
    g = torch.Generator().manual_seed(S)
    rows = {r for r in (0, 1, 31, 32, 63, 64, 127, 128, 255, 256, 257, S - 2, S - 1) if 0 <= r < S}
    rows |= set(torch.randint(0, S, (12,), generator=g).tolist())
    rows = torch.tensor(sorted(rows), device="cuda")
    some = {k: ops[k][:, rows] for k in ("x", "x2", "residual") if k in ops}
    R.check(out[:, rows], R.linear(**dict(ops, **some)), name)
