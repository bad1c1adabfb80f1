"""Cross-attention with scores far from 0 (some 2^34: q and k of 1e4, finite in bf16):
the largest key's weight is 1 however large its score.

Queries and keys are multiples of one vector of signs: q_i = c_i s, k_j = a_j s,
scale q_i . k_j = scale D c_i a_j. c and a have 8 significant bits, so that every
product and every partial sum of up to 128 equal ones (16 + 7 bits) is exact in
fp32. a takes few values, at least 2^-3 apart relative to the largest: scores that
differ do so by more than 2^20, far more than their own rounding (an ulp of 2^35 is
2^12), and weights are 0 but for the keys whose a is extreme, which tie. So a row is
the mean of their v: p = 1 each, sums of n terms in fp32 (n / 16 + 40 steps of
2^-22 of the magnitudes), one division and one rounding to bf16 (2^-8)."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _inputs(B, Sq, Sk, H, Hk, D, size, seed):
    g = torch.Generator().manual_seed(seed)
    signs = torch.randint(0, 2, (D,), generator=g).double() * 2 - 1
    # rows near +size and -size, whose extreme keys are the largest or the smallest a
    c = size * (1 + torch.randint(0, 128, (B, Sq, H), generator=g) / 128)
    c = c * (torch.randint(0, 2, (B, Sq, H), generator=g) * 2 - 1)
    a = size * torch.tensor([-1.75, -1.5, -1.25, 1.25, 1.5, 1.75])[
        torch.randint(0, 6, (B, Sk, Hk), generator=g)]
    q, k = c.double()[..., None] * signs, a.double()[..., None] * signs
    v = torch.randn(B, Sk, Hk, D, generator=g)
    q, k, v = (t.bfloat16() for t in (q, k, v))
    assert torch.equal(q.double(), c.double()[..., None] * signs)
    return q, k, v, c.double(), a.double()


def _want(c, a, v, keep):
    """(mean of v over the tied keys, bound), in 64 bits."""
    B, Sq, H = c.shape
    Hk = a.shape[2]
    ref = torch.zeros(B, Sq, H, v.shape[-1], dtype=torch.float64)
    bound = torch.zeros_like(ref)
    for b in range(B):
        if not keep[b].any():
            continue
        for h in range(H):
            aa, vv = a[b, keep[b], h * Hk // H], v[b, keep[b], h * Hk // H].double()
            z = c[b, :, h, None] * aa
            w = (z == z.amax(-1, keepdim=True)).double()
            w /= w.sum(-1, keepdim=True)
            r = w @ vv
            err = (len(aa) / 16 + 40) * 2.0 ** -22 * (w @ vv.abs())
            ref[b, :, h] = r
            bound[b, :, h] = err + 2.0 ** -8 * (r.abs() + err)
    return ref, bound + 2.0 ** -133


@pytest.mark.parametrize("size", [2.0 ** 13, 2.0 ** 14, 2.0 ** 30], ids=["2^33", "2^35", "2^67"])
@pytest.mark.parametrize("keys", ["all", "lengths", "mask"])
@pytest.mark.parametrize("B,Sq,Sk,H,Hk,D", [
    (2, 3, 300, 4, 2, 128),     # few queries: one CTA, keys over several
    (1, 2, 3000, 8, 8, 64),
    (1, 5, 6000, 24, 8, 128),
    (2, 900, 700, 16, 8, 128),  # many
    (2, 1300, 333, 6, 2, 64)])
def test_the_largest_keys_share_the_row(B, Sq, Sk, H, Hk, D, keys, size):
    q, k, v, c, a = _inputs(B, Sq, Sk, H, Hk, D, size, seed=Sk)
    keep = torch.ones(B, Sk, dtype=torch.bool)
    kw = {}
    if keys == "lengths":
        lengths = torch.tensor([Sk - 7, 130][:B], dtype=torch.int32)
        keep = torch.arange(Sk) < lengths[:, None]
        kw["lengths"] = lengths.cuda()
    if keys == "mask":
        keep = torch.rand(B, Sk, generator=torch.Generator().manual_seed(Sq)) < 0.6
        keep[:, :140] = False  # the first tile has no key
        kw["mask"] = keep.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.cross_attention(q.cuda(), k.cuda(), v.cuda(), status=status, **kw)
    got = got.cpu().double()
    assert int(status.item()) == 0
    want, bound = _want(c, a, v, keep)
    assert bool(got.isfinite().all())
    assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() - bound).max())
