"""binding.modulated_norm against the 64-bit definition."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _make(B, S, dim, y=True, gate=True, mod=True, x=BF, vec=BF, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(2000 + seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    ops = dict(x=(r(B, S, dim) * (0.5 + r(dim).abs()) + offset).to(x))
    mods = (0.5 * r(B, 3, dim)).to(vec).cuda()  # a modulation layer's output
    if mod:
        ops.update(shift=mods[:, 0], scale=mods[:, 1])
    if y:
        ops["y"] = r(B, S, dim).bfloat16()
        if gate:
            ops["gate"] = mods[:, 2]
    return {k: v.cuda() for k, v in ops.items()}


def _check(got, ops, what, **kw):
    h, xo = R.modulated_norm(**ops, **kw)
    torch.cuda.synchronize()
    if "y" in ops:
        R.check(got[0], h, what + " h")
        R.check(got[1], xo, what + " x_out")
        assert got[1].dtype == ops["x"].dtype
    else:
        R.check(got, h, what)


# every width class of the kernel and both sides of its borders
@pytest.mark.parametrize("dim", [8, 16, 120, 256, 264, 504, 512, 520, 1024, 1032, 2048, 2056, 4096,
                                 4104, 6144, 6152, 8192, 8200, 16384])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_widths(dim, kind):
    for i, (x, vec, y) in enumerate(((BF, BF, False), (F32, F32, True), (BF, F32, True))):
        ops = _make(2, 5, dim, y=y, x=x, vec=vec, seed=dim + i)
        _check(binding.modulated_norm(**ops, norm=kind), ops, f"{dim} {kind} {x}", norm=kind)


@pytest.mark.parametrize("B,S,dim", [(1, 1, 8), (1, 1, 4096), (3, 1, 72), (1, 7, 512), (2, 333, 264),
                                     (5, 41, 1000), (1, 2000, 320)])
@pytest.mark.parametrize("form", [dict(y=False, mod=False), dict(y=False), dict(gate=False),
                                  dict(mod=False), dict(x=F32, vec=F32), dict(vec=F32)])
def test_forms(B, S, dim, form):
    ops = _make(B, S, dim, **form, seed=S)
    _check(binding.modulated_norm(**ops), ops, f"{B}x{S}x{dim} {form}")


def test_large_mean_small_spread_and_constant_rows():
    """The variance is taken about the mean; a constant row has variance 0 and
    is eps' to scale."""
    ops = _make(1, 6, 1000, y=False, x=F32, vec=F32, offset=300.0)
    _check(binding.modulated_norm(**ops), ops, "offset")
    x = torch.full((1, 3, 512), 5.0, device="cuda")
    x[0, 1] = 0
    h = binding.modulated_norm(x, shift=torch.full((512,), 0.25, device="cuda"))
    assert bool((h == 0.25).all())
    x = torch.full((1, 2, 64), 1e-4, device="cuda")
    ops = dict(x=x)
    for eps in (0.0, 1e-6, 1.0):
        _check(binding.modulated_norm(**ops, norm="rms", eps=eps), ops, "eps", norm="rms", eps=eps)


@pytest.mark.parametrize("x", [BF, F32])
@pytest.mark.parametrize("B,S,dim", [(2, 9, 136), (1, 300, 520), (3, 1, 64)])
def test_views_and_what_lies_around_them(B, S, dim, x):
    ops = _make(B, S, dim, x=x, vec=F32, seed=S)
    for name in ("x", "y"):
        buf = torch.full((B, S + 3, dim + 24), float("nan"), dtype=ops[name].dtype, device="cuda")
        buf[:, 3:, 8:-16] = ops[name]
        ops[name] = buf[:, 3:, 8:-16]
    bufs = [torch.full((B, S + 4, dim + 16), 7.0, dtype=t, device="cuda") for t in (BF, x)]
    h, xo = (b[:, 2:-2, 8:-8] for b in bufs)
    got = binding.modulated_norm(**ops, out=h, x_out=xo)
    assert got[0] is h and got[1] is xo
    _check(got, ops, "views")
    for b in bufs:
        inner = b[:, 2:-2, 8:-8].clone()
        b[:, 2:-2, 8:-8] = 7.0
        assert bool((b == 7.0).all())
        b[:, 2:-2, 8:-8] = inner
    # [S, B, dim] storage
    ops["x"] = ops["x"].transpose(0, 1).contiguous().transpose(0, 1)
    _check(binding.modulated_norm(**ops), ops, "token major")


@pytest.mark.parametrize("x", [BF, F32])
def test_in_place_and_repeatable(x):
    ops = _make(2, 77, 776, x=x, vec=F32)
    h, xo = binding.modulated_norm(**ops)
    h2, xo2 = binding.modulated_norm(**ops, x_out=ops["x"])
    assert xo2 is ops["x"] and torch.equal(xo, xo2) and torch.equal(h, h2)


def test_rows_do_not_mix():
    """NaN and infinities stay in their row, also where rows share a block."""
    for dim in (64, 520, 1032, 4096):
        ops = _make(1, 20, dim)
        h, xo = (t.clone() for t in binding.modulated_norm(**ops))
        bad = ops["x"].clone()
        bad[0, 3, 5] = float("nan")
        bad[0, 11] = float("inf")
        bad[0, 12, 0] = torch.finfo(BF).min
        h2, xo2 = binding.modulated_norm(**dict(ops, x=bad))
        keep = [s for s in range(20) if s not in (3, 11, 12)]
        assert torch.equal(h[0, keep], h2[0, keep]) and torch.equal(xo[0, keep], xo2[0, keep])
        assert bool(torch.isnan(h2[0, 3]).all())


def test_broadcast_vectors_and_two_dimensions():
    ops = _make(3, 4, 136)
    vecs = ("scale", "shift", "gate")
    one = {k: ops[k][0].contiguous() for k in vecs}
    want = binding.modulated_norm(**dict(ops, **{k: v.expand(3, 136).contiguous()
                                                 for k, v in one.items()}))
    for got in (binding.modulated_norm(**dict(ops, **one)),
                binding.modulated_norm(**dict(ops, **{k: v.expand(3, 136) for k, v in one.items()}))):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    flat = binding.modulated_norm(**dict(ops, x=ops["x"][0], y=ops["y"][0], **one))
    assert flat[0].shape == (4, 136) and torch.equal(flat[0], want[0][0])


def test_on_another_stream_and_in_a_graph():
    ops = _make(2, 50, 520, x=F32, vec=F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.modulated_norm(**ops, stream=side)
    side.synchronize()
    _check(got, ops, "side stream")
    out, x_out = torch.empty_like(got[0]), torch.empty_like(got[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.modulated_norm(**ops, out=out, x_out=x_out)
    other = _make(2, 50, 520, x=F32, vec=F32, seed=1)
    for k in ops:
        ops[k].copy_(other[k])
    graph.replay()
    _check((out, x_out), ops, "graph")


def test_offsets_past_32_bits():
    S, dim = 300_000, 8192
    x = torch.empty(1, S, dim, dtype=BF, device="cuda").normal_(generator=torch.Generator(
        device="cuda").manual_seed(4))
    h = binding.modulated_norm(x)
    rows = torch.tensor([0, 131_072, 262_143, 262_144, S - 1], device="cuda")
    R.check(h[:, rows], R.modulated_norm(x[:, rows])[0], "far rows")


def test_refusals():
    ops = _make(2, 5, 64)
    for kw in (dict(norm="batch"), dict(x=ops["x"].half()), dict(y=ops["y"].float()),
               dict(y=ops["y"][:, :4]), dict(scale=ops["scale"].float()),
               dict(shift=ops["shift"][:, :32]), dict(gate=ops["gate"].cpu()),
               dict(x=ops["x"].cpu()), dict(x=ops["x"][..., ::2]), dict(y=None),
               dict(x_out=ops["x"].float())):
        with pytest.raises(ValueError):
            binding.modulated_norm(**dict(ops, **kw))
    plain = {k: ops[k] for k in ("x", "scale", "shift")}
    for kw, code in ((dict(out=ops["x"]), -9), (dict(eps=-1.0), -2),
                     (dict(x=ops["x"][:1].expand(2, 5, 64)), -2)):
        with pytest.raises(binding.FluxError) as e:
            binding.modulated_norm(**dict(plain, **kw))
        assert e.value.status == code
    odd = torch.zeros(2, 5, 60, device="cuda").bfloat16()
    with pytest.raises(binding.FluxError):
        binding.modulated_norm(odd)
