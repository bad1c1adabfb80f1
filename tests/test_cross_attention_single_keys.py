"""Cross-attention whose rows are each decided by one key: a query is four times a key
at an edge (of a tile, of a word of 32 keys, of a CTA's part of the keys, of a length),
so that its weight is all but 1 and the row that key's v. A key that is lost, counted
for another, or taken in although it is left out, changes a whole row, where one key
among thousands of alike weights hides behind the weights' rounding."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R
from tests import cross_reference as X
from tests import operator_cases as C


def _edges(Sk, length, parts):
    """Keys on both sides of every edge of `length` of Sk keys in `parts` parts."""
    n = -(-length // 128)
    at = {0, length, Sk}
    at |= {128 * (n * p // parts) for p in range(parts + 1)}
    at |= set(range(128, Sk, 128)) if Sk < 2000 else {128, 256, 128 * (n // 2), 128 * (n - 1)}
    at |= {32, 96, 128 + 64, Sk - Sk % 128 + 32}
    return sorted({j for e in at for j in (e - 2, e - 1, e, e + 1) if 0 <= j < Sk})


def _queries(k, at, H):
    """[B, Sq, H, D]: four times the keys `at` [B, Sq, H] of the heads' key heads."""
    B, Sq = at.shape[:2]
    head = (torch.arange(H) * k.shape[2] // H).expand(Sq, H)
    return torch.stack([4 * k[b][at[b], head].float() for b in range(B)]).bfloat16(), head


@pytest.mark.parametrize("D", [64, 128])
def test_a_lost_key_shows(D):
    """On the reference: without its key, or with a neighbour's v, every row is far
    outside the bound that the kernel is held to."""
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn(1, 6000, 1, D, generator=g).bfloat16() for _ in "kv")
    at = torch.tensor([0, 127, 128, 639, 640, 5999]).reshape(1, 6, 1)
    q, _ = _queries(k, at, 1)
    want, bound = X.cross(q, k, v)
    for i, j in enumerate(at[0, :, 0].tolist()):
        lost = torch.ones(1, 6000, dtype=torch.bool)
        lost[0, j] = False
        for bad in (X.cross(q, k, v, mask=lost)[0], X.cross(q, k, v.roll(1, 1))[0]):
            assert bool(((bad - want)[0, i].abs() > 4 * bound[0, i]).float().mean() > 0.9)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("keys", ["all", "lengths", "mask", "both"])
@pytest.mark.parametrize("key", list(C.CROSS))
def test_rows_of_one_key(key, keys, D):
    build.build()
    B, Sq, Sk, H, Hk, _ = C.CROSS[key]
    parts = key[1]
    g = torch.Generator().manual_seed(Sq + Sk + D)
    k, v = (torch.randn(B, Sk, Hk, D, generator=g).bfloat16() for _ in "kv")
    kw, lengths = {}, [Sk] * B
    if keys in ("lengths", "both"):
        lengths = [Sk - 3, Sk // 2 + 1][:B]
        kw["lengths"] = torch.tensor(lengths, dtype=torch.int32)
    if keys in ("mask", "both"):
        kw["mask"] = torch.rand(B, Sk, generator=g) < 0.8
    dev = {n: t.cuda() for n, t in kw.items()}
    kd, vd = k.cuda(), v.cuda()
    edges = [_edges(Sk, n, parts) for n in lengths]
    rows = Sq * H
    calls = max(-(-len(e) // rows) for e in edges)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in range(calls):
        # queries of a call take the edges in turn, heads first
        at = torch.stack([torch.tensor([e[(call * rows + i) % len(e)] for i in range(rows)])
                          .reshape(Sq, H) for e in edges])
        q, head = _queries(k, at, H)
        got = binding.cross_attention(q.cuda(), kd, vd, status=status, **dev)
        assert int(status.item()) == 0
        some = torch.arange(Sq)[:max(1, -(-max(map(len, edges)) // H))]  # each edge once or more
        R.check(got[:, some.cuda()], X.cross(q[:, some], k, v, **kw), f"{key} {keys} {call}")
        # All rows: one key's v, where that key takes part. (Its exponent 4 |k|^2 / sqrt(D) is
        # 32 on average at D = 64, the others' 4 at the root of their mean square: together
        # they weigh some 2^-11, and up to 2^-6 where |k|^2 is a third of its mean.)
        for b in range(B):
            keep = torch.arange(Sk) < lengths[b]
            keep &= kw["mask"][b] if "mask" in kw else True
            want = v[b][at[b], head].float()
            near = ((got[b].cpu().float() - want).abs() <= 2.0 ** -5 * (1 + want.abs())).all(-1)
            assert bool(near[keep[at[b]]].all())
