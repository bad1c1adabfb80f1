"""binding.cross_attention against the definition in 64 bits: few and many
queries, one key to long documents, shared heads, lengths and masks, views."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R
from tests import cross_reference as X

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _make(B, Sq, Sk, H, Hk, D, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(7000 + seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k, v = spread * r(B, Sq, H, D), r(B, Sk, Hk, D), r(B, Sk, Hk, D)
    return dict(q=q.bfloat16().cuda(), k=k.bfloat16().cuda(), v=v.bfloat16().cuda())


def _run(ops, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.cross_attention(status=status, **ops, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out


SIZES = [
    (1, 1, 1, 1, 1, 128),           # the smallest call
    (1, 1, 1, 1, 1, 64),
    (1, 3, 129, 2, 2, 64),
    (2, 1, 77, 4, 4, 128),
    (1, 64, 1000, 3, 3, 128),       # keys over several CTAs, two streams each
    (1, 1, 5000, 8, 2, 128),        # one token, a group of four heads
    (2, 5, 2050, 6, 2, 64),         # groups of three
    (1, 130, 300, 2, 2, 128),
    (1, 257, 513, 5, 1, 64),        # groups of five, ragged tiles
    (3, 300, 77, 4, 4, 128),
    (1, 1500, 260, 7, 7, 128),
    (2, 2200, 130, 16, 8, 128),     # many queries: more items than SMs
    (1, 4000, 90, 24, 24, 64),
    (1, 9, 40, 128, 1, 64),         # a group as large as a tile
]


@pytest.mark.parametrize("B,Sq,Sk,H,Hk,D", SIZES)
def test_sizes(B, Sq, Sk, H, Hk, D):
    ops = _make(B, Sq, Sk, H, Hk, D)
    R.check(_run(ops), X.cross(**ops), f"{B} {Sq} {Sk} {H} {Hk} {D}")


@pytest.mark.parametrize("B,Sq,Sk,H,Hk,D", [
    (4, 40, 700, 2, 2, 128), (4, 1, 3000, 4, 1, 64), (5, 700, 300, 8, 8, 128), (4, 900, 400, 6, 2, 64)])
@pytest.mark.parametrize("kind", ["lengths", "mask", "both"])
def test_keys_left_out(B, Sq, Sk, H, Hk, D, kind):
    """Lengths from none to all (and outside that), masks that leave out tiles, a
    batch element, all but one key; what lies there is NaN and infinite."""
    ops = _make(B, Sq, Sk, H, Hk, D, seed=Sk)
    g = torch.Generator().manual_seed(Sk)
    lengths = torch.tensor([0, Sk + 5, 1, 129, -3][:B], dtype=torch.int32)
    mask = torch.rand(B, Sk, generator=g) < 0.7
    mask[1] = False
    mask[1, Sk - 2] = True
    mask[2, :256] = False
    mask[3] = False
    keep = torch.ones(B, Sk, dtype=torch.bool)
    kw = {}
    if kind != "mask":
        keep &= torch.arange(Sk) < lengths[:, None]
        kw["lengths"] = lengths.cuda()
    if kind != "lengths":
        keep &= mask
        kw["mask"] = mask.cuda()
    want = X.cross(**ops, **{n: t.cpu() for n, t in kw.items()})
    out = keep.logical_not().cuda()
    for name, bad in (("k", float("nan")), ("v", float("inf"))):
        ops[name][out] = bad
        ops[name][out.roll(1, 1) & out] = float("nan")
    got = _run(ops, **kw)
    R.check(got, want, kind)
    assert bool((got[~keep.any(1).cuda()] == 0).all())


@pytest.mark.parametrize("Sq", [3, 1300])
def test_mask_bytes_shared_by_the_batch_and_unaligned(Sq):
    ops = _make(3, Sq, 333, 4, 4, 128, seed=5)
    buf = torch.zeros(340, dtype=torch.uint8)
    buf[5:338] = torch.arange(333) % 3 == 0
    buf[5:338] *= 7
    mask = buf.cuda()[5:338].expand(3, 333)
    R.check(_run(ops, mask=mask), X.cross(**ops, mask=mask), "bytes")


@pytest.mark.parametrize("B,Sq,Sk,H,Hk,D", [(2, 7, 900, 4, 2, 128), (2, 700, 140, 4, 4, 64),
                                            (2, 500, 200, 6, 2, 128)])
def test_views(B, Sq, Sk, H, Hk, D):
    """q inside a joint sequence, k and v side by side, out in a wider buffer: what
    lies around it is left as it was."""
    ops = _make(B, Sq, Sk, H, Hk, D, seed=9)
    want = X.cross(**ops)
    nan = float("nan")
    qbuf = torch.full((B, Sq + 9, 2 * H, D), nan, dtype=torch.bfloat16, device="cuda")
    qbuf[:, 9:, H:] = ops["q"]
    kv = torch.full((B, Sk + 3, 2, Hk, D), nan, dtype=torch.bfloat16, device="cuda")
    kv[:, :Sk, 0], kv[:, :Sk, 1] = ops["k"], ops["v"]
    obuf = torch.full((B, Sq + 4, H + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out = obuf[:, 2:-2, 1:-1]
    got = _run(dict(q=qbuf[:, 9:, H:], k=kv[:, :Sk, 0], v=kv[:, :Sk, 1]), out=out)
    assert got is out
    R.check(out, want, "views")
    assert bool((obuf[:, :2] == 7).all() and (obuf[:, -2:] == 7).all())
    assert bool((obuf[:, :, 0] == 7).all() and (obuf[:, :, -1] == 7).all())


@pytest.mark.parametrize("Sq", [2, 900])
def test_large_scores_and_scale(Sq):
    """Scores that grow along the keys, so that the running maximum rises by more
    than a rescale's threshold in every tile, and a scale of the caller's."""
    ops = _make(1, Sq, 1100, 4, 4, 128, seed=3)
    ramp = torch.linspace(0.1, 6.0, 1100, device="cuda")[None, :, None, None]
    ops["k"] = (ops["k"].float() * ramp).bfloat16()
    R.check(_run(ops, scale=0.3), X.cross(**ops, scale=0.3), "ramp")
    ops["k"] = ops["k"].flip(1).contiguous()
    R.check(_run(ops, scale=0.3), X.cross(**ops, scale=0.3), "falling")


@pytest.mark.parametrize("Sq,Sk", [(1, 4000), (1200, 300)])
def test_the_same_call_gives_the_same_bits(Sq, Sk):
    ops = _make(2, Sq, Sk, 8, 4, 128)
    a, b = _run(ops), _run(ops)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_nan_in_a_query_stays_in_its_row():
    ops = _make(1, 300, 200, 2, 2, 128)
    ops["q"][0, 17, 1, 5] = float("nan")
    got = _run(ops)
    assert got[0, 17, 1].isnan().all()
    got[0, 17, 1] = 0
    ops["q"][0, 17, 1, 5] = 0
    want, bound = X.cross(**ops)
    want[0, 17, 1] = 0
    R.check(got, (want, bound + 2.0 ** -133), "the other rows")


@pytest.mark.parametrize("Sq,D", [(42, 128), (42, 64), (3000, 128), (3000, 64)])
def test_what_an_earlier_call_left_does_not_show(Sq, D):
    """Groups of three fill 126 of a tile's 128 rows: whatever the call before had
    in the other two, the bits are the same."""
    ops = _make(2, Sq, 1000, 6, 2, D)
    before = _make(1, 40000, 300, 1, 1, D, spread=300.0)  # every SM's query tiles
    _run(before)
    a = _run(ops)
    before["q"].zero_()
    _run(before)
    b = _run(ops)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("B,Sq,Sk,H,Hk,D", [
    (1, 7, 300, 100, 1, 64),      # a query's heads fill 100 of a tile's rows
    (2, 300, 200, 66, 2, 128),    # groups of 33, three queries a tile
    (1, 3, 4000, 127, 1, 128),    # keys over several CTAs
    (1, 900, 129, 65, 1, 64)])
def test_groups_that_do_not_fill_a_tile(B, Sq, Sk, H, Hk, D):
    ops = _make(B, Sq, Sk, H, Hk, D, seed=H)
    R.check(_run(ops), X.cross(**ops), f"{H} over {Hk}")


@pytest.mark.parametrize("B,Sq,Sk,H,Hk,D", [(2, 1, 4000, 8, 2, 128), (3, 40, 100, 4, 4, 64),
                                            (2, 3000, 300, 8, 8, 128), (1, 2000, 700, 3, 1, 64)])
@pytest.mark.parametrize("kind", ["lengths", "mask", "both"])
def test_no_key_for_anybody(B, Sq, Sk, H, Hk, D, kind):
    ops = _make(B, Sq, Sk, H, Hk, D)
    for name in ("k", "v"):
        ops[name].fill_(float("nan"))
    kw = {}
    if kind != "mask":
        kw["lengths"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if kind != "lengths":
        kw["mask"] = torch.zeros(B, Sk, dtype=torch.bool, device="cuda")
    out = torch.full((B, Sq, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    assert bool((_run(ops, out=out, **kw) == 0).all())
