"""flux_quantize_fp8, flux_linear_fp8 and flux_cross_attention on the host: bad
arguments are refused with the documented status before a device is touched, and
the references that the GPU tests use agree with independent forms."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import cross_reference as X
from tests import fp8_reference as F

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _on_device(rc):
    """Every host check passed: the call got as far as the device check (this
    process has no sm_103 device), or ran."""
    return rc in (0, -6, -8)


QUANTIZE = dict(x=256 * MB, x_bs=25600, x_rs=256, x_f32=0, B=2, S=100, K=256, rows=1, q=512 * MB,
                q_bs=25600, q_rs=256, scale=600 * MB, s_bs=100, s_rs=1, s_ks=200)
LINEAR = dict(x=256 * MB, x_bs=25600, x_rs=256, xs=300 * MB, xs_bs=100, xs_rs=1, xs_ks=200,
              w=512 * MB, w_rs=256, ws=600 * MB, ws_rs=2, ws_ks=1, B=2, S=100, K=256, N=128, act=0,
              bias=None, gate=None, gate_bs=0, vec_f32=0, residual=None, r_bs=0, r_rs=0,
              out=1024 * MB, o_bs=12800, o_rs=128, status=2048 * MB)
CROSS = dict(q=256 * MB, q_bs=51200, q_rs=512, k=300 * MB, k_bs=25600, k_rs=256, v=400 * MB,
             v_bs=25600, v_rs=256, lengths=None, mask=None, mask_bs=0, B=2, Sq=100, Sk=100, H=4,
             Hk=2, D=128, scale=0.0, out=1024 * MB, o_bs=51200, o_rs=512, status=2048 * MB)
CALLS = {"flux_quantize_fp8": QUANTIZE, "flux_linear_fp8": LINEAR, "flux_cross_attention": CROSS}


def _call(lib, name, kw):
    a = dict(CALLS[name], **kw)
    assert len(a) == len(CALLS[name])
    return getattr(lib, name)(*a.values(), None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses stay off a GPU")
@pytest.mark.parametrize("name,kw", [
    ("flux_quantize_fp8", {}), ("flux_quantize_fp8", dict(x_f32=1)),
    ("flux_quantize_fp8", dict(rows=128, B=1, s_rs=2, s_ks=1)),
    ("flux_quantize_fp8", dict(s_bs=200, s_rs=2, s_ks=1)),
    ("flux_quantize_fp8", dict(B=1, S=1, x_rs=3, q_rs=5, x_bs=-1, s_rs=0, s_bs=-7)),  # not looked at
    ("flux_quantize_fp8", dict(K=128, x_rs=128, x_bs=12800, s_ks=-3)),
    ("flux_linear_fp8", {}), ("flux_linear_fp8", dict(xs_bs=0, xs_rs=0, xs_ks=0, ws_rs=0, ws_ks=0)),
    ("flux_linear_fp8", dict(residual=1024 * MB, r_bs=12800, r_rs=128)),          # in place
    ("flux_linear_fp8", dict(act=3)), ("flux_linear_fp8", dict(N=8, o_rs=8, o_bs=800)),
    ("flux_linear_fp8", dict(K=16, x_rs=16, w_rs=16, x_bs=1600)),
    ("flux_linear_fp8", dict(o_rs=256, o_bs=128)),                                # [S, B, N]
    ("flux_cross_attention", {}), ("flux_cross_attention", dict(lengths=900 * MB, mask=901 * MB + 3)),
    ("flux_cross_attention", dict(v=300 * MB + 512, k_rs=512, v_rs=512, k_bs=51200, v_bs=51200)),
    ("flux_cross_attention", dict(D=64, scale=2.0)), ("flux_cross_attention", dict(H=256, Hk=2, D=64,
                                                                                   q_rs=16384, o_rs=16384,
                                                                                   q_bs=1638400,
                                                                                   o_bs=1638400)),
    ("flux_cross_attention", dict(mask=900 * MB, mask_bs=0)),
])
def test_accepts(lib, name, kw):
    assert _on_device(_call(lib, name, kw))


@pytest.mark.parametrize("name,kw,code", [
    *[("flux_quantize_fp8", {k: None}, -1) for k in ("x", "q", "scale")],
    *[("flux_linear_fp8", {k: None}, -1) for k in ("x", "xs", "w", "ws", "out", "status")],
    *[("flux_cross_attention", {k: None}, -1) for k in ("q", "k", "v", "out", "status")],
    *[("flux_quantize_fp8", kw, -2) for kw in (
        dict(B=0), dict(S=0), dict(S=-1), dict(B=1 << 20, S=1 << 20), dict(K=0), dict(K=8),
        dict(K=250), dict(K=(1 << 22) + 16), dict(rows=2), dict(rows=0), dict(rows=128),  # B = 2
        dict(x_f32=2), dict(x_rs=248), dict(x_rs=260), dict(q_rs=264), dict(q_bs=0), dict(q_rs=-256),
        dict(s_rs=-1), dict(s_rs=0), dict(s_ks=100), dict(s_bs=1), dict(x_bs=1 << 62))],
    *[("flux_linear_fp8", kw, -2) for kw in (
        dict(B=0), dict(S=0), dict(K=0), dict(K=100), dict(K=8), dict(N=0), dict(N=100), dict(act=4),
        dict(act=-1), dict(act=3, N=64, o_rs=64, o_bs=6400), dict(vec_f32=2), dict(x_rs=240),
        dict(x_rs=264), dict(x_bs=8), dict(w_rs=264), dict(w_rs=128), dict(xs_rs=-1), dict(ws_ks=-1),
        dict(xs_ks=1 << 62), dict(o_bs=6400), dict(o_rs=132), dict(gate=700 * MB, gate_bs=-8),
        dict(B=1 << 20, S=1 << 20))],
    *[("flux_cross_attention", kw, -2) for kw in (
        dict(B=0), dict(Sq=0), dict(Sk=0), dict(H=0), dict(Hk=0), dict(Hk=3), dict(H=258, Hk=2),
        dict(D=96), dict(D=32), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
        dict(q_rs=504), dict(q_rs=514), dict(k_rs=128), dict(v_bs=0), dict(o_bs=256),
        dict(mask=900 * MB, mask_bs=-1), dict(B=1 << 20, Sq=1 << 20),
        dict(Sq=1 << 30, B=1, H=32, Hk=32, q_rs=4096, o_rs=4096))],
    *[("flux_quantize_fp8", kw, -4) for kw in (dict(x=256 * MB + 8), dict(q=512 * MB + 8),
                                               dict(scale=600 * MB + 2))],
    *[("flux_linear_fp8", kw, -4) for kw in (
        dict(x=256 * MB + 8), dict(w=512 * MB + 8), dict(out=1024 * MB + 8), dict(xs=300 * MB + 2),
        dict(ws=600 * MB + 1), dict(bias=700 * MB + 8), dict(gate=700 * MB + 4), dict(status=2048 * MB + 2),
        dict(residual=800 * MB + 8, r_bs=12800, r_rs=128))],
    *[("flux_cross_attention", kw, -4) for kw in (
        dict(q=256 * MB + 8), dict(k=300 * MB + 2), dict(v=400 * MB + 8), dict(out=1024 * MB + 8),
        dict(lengths=900 * MB + 2), dict(status=2048 * MB + 1))],
    *[("flux_quantize_fp8", kw, -9) for kw in (
        dict(q=256 * MB), dict(scale=256 * MB + 64), dict(scale=512 * MB + 64))],
    *[("flux_linear_fp8", kw, -9) for kw in (
        dict(out=256 * MB), dict(out=512 * MB), dict(xs=1024 * MB + 64), dict(ws=1024 * MB + 64),
        dict(bias=1024 * MB + 64), dict(gate=1024 * MB + 64), dict(status=1024 * MB + 64),
        dict(residual=1024 * MB + 256, r_bs=12800, r_rs=128))],
    *[("flux_cross_attention", kw, -9) for kw in (
        dict(out=256 * MB), dict(out=300 * MB), dict(out=400 * MB), dict(lengths=1024 * MB + 64),
        dict(mask=1024 * MB + 65), dict(status=1024 * MB + 64))],
])
def test_refuses(lib, name, kw, code):
    assert _call(lib, name, kw) == code


@pytest.mark.parametrize("call", [
    lambda t: binding.quantize_fp8(t), lambda t: binding.linear_fp8(t, t, t, t),
    lambda t: binding.cross_attention(t[None, None], t[None, None], t[None, None])])
def test_cpu_tensors_are_refused(lib, call):
    with pytest.raises(ValueError):
        call(torch.zeros(16, 128, dtype=torch.bfloat16))


def test_e4m3_reference_rounds_to_the_nearest():
    """Against every e4m3 value: the chosen one is as near as any (half a step)."""
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = every[every.isfinite()]
    x = torch.randn(4, 256, generator=torch.Generator().manual_seed(1)) * 3
    q, s = F.quantize(x)
    scaled = (x * (448.0 / (s * 448)).repeat_interleave(128, 1)).double()
    gap = (scaled[..., None] - every).abs().amin(-1)
    # (the factor is rounded once more than here: relative 2^-22 of at most 448)
    assert bool(((q.double() - scaled).abs() <= gap + 448 * 2.0 ** -22).all())
    assert bool((q.double().abs().reshape(4, 2, 128).amax(-1) == 448).all())


def test_cross_reference_agrees_with_a_loop():
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(2, n, h, 64, generator=g).bfloat16() for n, h in ((3, 4), (9, 2), (9, 2)))
    lengths, mask = torch.tensor([0, 7]), torch.rand(2, 9, generator=g) < 0.5
    ref, bound = X.cross(q, k, v, lengths, mask)
    for b in range(2):
        for i in range(3):
            for h in range(4):
                keys = [j for j in range(9) if j < lengths[b] and mask[b, j]]
                if not keys:
                    assert bool((ref[b, i, h] == 0).all())
                    continue
                w = [float(torch.exp(q[b, i, h].double() @ k[b, j, h // 2].double() / 8)) for j in keys]
                want = sum(x * v[b, j, h // 2].double() for x, j in zip(w, keys)) / sum(w)
                assert bool(((ref[b, i, h] - want).abs() < 1e-12).all())
    assert bool((bound[1] > 0).all() and (bound < 0.1).all())
