"""binding.modulated_norm where a group of warps walks many rows: across batch
elements with vectors of their own, steps that pass whole batch elements, views,
and updates in place, every row against the 64-bit definition."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# Batch, tokens, channels. On 152 SMs a group of warps gets the row, the row 152
# (304, ...) further and so on: 14 rows and two changes of the batch element; 15
# and one, ragged channels; steps of a few batch elements and a rest of one;
# several groups per block, steps of many batch elements.
SIZES = [(3, 700, 4096), (2, 1100, 4104), (60, 40, 1032), (400, 7, 520)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _make(B, S, dim, x, vec, y, views, seed):
    """Operands of which every batch element's vectors differ in size and sign."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ops = dict(x=(r(B, S, dim) * (0.5 + r(dim).abs()) + r(B, S, 1)).to(x))
    mods = ((0.3 + torch.arange(B, device="cuda")[:, None, None] % 5) * r(B, 3, dim)).to(vec)
    ops.update(shift=mods[:, 0], scale=mods[:, 1])
    if y:
        ops.update(y=r(B, S, dim).bfloat16(), gate=mods[:, 2])
    if views:  # rows and channels inside wider buffers
        for name in ("x", "y"):
            if name in ops:
                t = ops[name]
                buf = torch.full((B, S + 3, dim + 24), float("nan"), dtype=t.dtype, device="cuda")
                buf[:, 2:-1, 16:-8] = t
                ops[name] = buf[:, 2:-1, 16:-8]
    return ops


@pytest.mark.parametrize("B,S,dim", SIZES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("x,vec,y", [(BF, BF, False), (BF, BF, True), (BF, F32, True),
                                     (F32, F32, True), (F32, BF, True), (F32, F32, False)])
def test_many_rows_of_many_batch_elements(B, S, dim, kind, x, vec, y):
    ops = _make(B, S, dim, x, vec, y, views=y, seed=dim + B)
    (h, hb), ref_x = R.modulated_norm(**ops, norm=kind)
    bufs = [torch.full((B, S + 2, dim + 16), 7.0, dtype=t, device="cuda") for t in (BF, x)]
    views = [b[:, 1:-1, 8:-8] for b in bufs]
    got = binding.modulated_norm(**ops, norm=kind, out=views[0], x_out=views[1] if y else None)
    torch.cuda.synchronize()
    R.check(views[0], (h, hb), "h")
    if y:
        assert got[1] is views[1]
        R.check(views[1], ref_x, "x_out")
    first = [v.clone() for v in views]
    for b, v in zip(bufs, views):
        v.fill_(7.0)
        assert bool((b == 7.0).all())
    if y:  # in place, and the same bits
        h2, xo = binding.modulated_norm(**ops, norm=kind, x_out=ops["x"])
        assert xo is ops["x"]
        assert torch.equal(h2, first[0]) and torch.equal(xo, first[1])
