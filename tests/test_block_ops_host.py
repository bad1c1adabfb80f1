"""flux_linear and flux_modulated_norm on the host: bad arguments are refused
with the documented status before a device is touched, overlap is judged by
elements where strides are equal, and the 64-bit references that the GPU tests
use agree with independent forms."""
import ctypes

import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _on_device(rc):
    """Every host check passed: the call got as far as the device check (this
    process has no sm_103 device), or ran."""
    return rc in (0, -6, -8)


LINEAR = dict(x=256 * MB, x_bs=64 * 100, x_rs=64, K=64, x2=None, x2_bs=0, x2_rs=0, K2=0,
              w=512 * MB, w_rs=64, B=2, S=100, N=128, act=0, bias=None, gate=None, gate_bs=0,
              vec_f32=0, residual=None, r_bs=0, r_rs=0, out=1024 * MB, o_bs=128 * 100, o_rs=128,
              status=2048 * MB)


def _linear(lib, **kw):
    a = dict(LINEAR, **kw)
    return lib.flux_linear(*[a[k] for k in LINEAR], None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses stay off a GPU")
@pytest.mark.parametrize("kw", [
    {},
    dict(residual=1024 * MB, r_bs=128 * 100, r_rs=128),              # in place
    dict(B=1, x_bs=-5, o_bs=0),                                      # not looked at
    dict(S=1, x_rs=3, o_rs=0, x_bs=64, o_bs=128),                    # not looked at
    dict(o_rs=256, o_bs=128),                                        # [S, B, N]
    dict(x=1024 * MB + 2 * 128, x_rs=192, x_bs=19200, o_rs=192, o_bs=19200),  # columns of one buffer
    dict(o_bs=256 * 100, x=1024 * MB + 2 * 128 * 100, x_bs=256 * 100, x_rs=128, K=128, w_rs=128),
    dict(gate=600 * MB, gate_bs=0), dict(gate=600 * MB, gate_bs=128),
    dict(w_rs=256), dict(act=3),
    dict(K2=64, x2=700 * MB, x2_rs=64, x2_bs=6400, w_rs=128),
])
def test_linear_accepts(lib, kw):
    assert _on_device(_linear(lib, **kw))


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(out=None), -1), (dict(status=None), -1),
    (dict(K2=64, w_rs=128), -1),
    (dict(B=0), -2), (dict(S=0), -2), (dict(S=-4), -2), (dict(B=1 << 20, S=1 << 20), -2),
    (dict(K=0), -2), (dict(K=60), -2), (dict(K2=-8), -2), (dict(N=0), -2), (dict(N=100), -2),
    (dict(act=4), -2), (dict(act=-1), -2), (dict(vec_f32=2), -2),
    (dict(x_rs=56), -2),             # rows overlap
    (dict(x_rs=68), -2),             # not a multiple of 8
    (dict(x_bs=0), -2), (dict(x_rs=0), -2), (dict(x_rs=-64), -2),
    (dict(x_rs=1 << 62), -2), (dict(x_bs=1 << 62), -2),
    (dict(o_bs=128 * 50), -2),       # the outputs' batch elements overlap
    (dict(w_rs=56), -2),
    (dict(gate=600 * MB, gate_bs=-128), -2), (dict(gate=600 * MB, gate_bs=129), -2),
    (dict(x=256 * MB + 8), -4), (dict(w=512 * MB + 2), -4), (dict(out=1024 * MB + 4), -4),
    (dict(bias=600 * MB + 4), -4), (dict(gate=600 * MB + 8), -4), (dict(status=2048 * MB + 2), -4),
    (dict(residual=700 * MB + 2, r_bs=12800, r_rs=128), -4),
    (dict(out=256 * MB), -9),        # x
    (dict(out=512 * MB), -9),        # w
    (dict(bias=1024 * MB + 1024), -9),
    (dict(gate=1024 * MB + 1024, gate_bs=128), -9),
    (dict(status=1024 * MB + 64), -9),
    (dict(residual=1024 * MB + 256, r_bs=12800, r_rs=128), -9),     # shifted by a row
    (dict(residual=1024 * MB, r_bs=12800 * 2, r_rs=256), -9),       # in place, other strides
    (dict(x=1024 * MB + 2 * 120, x_rs=192, x_bs=19200, o_rs=192, o_bs=19200), -9),  # 8 columns
])
def test_linear_refuses(lib, kw, code):
    assert _linear(lib, **kw) == code


NORM = dict(x=256 * MB, x_bs=6400, x_rs=64, stream_f32=0, y=None, y_bs=0, y_rs=0, gate=None,
            gate_bs=0, scale=None, scale_bs=0, shift=None, shift_bs=0, vec_f32=0, B=2, S=100,
            dim=64, norm=0, eps=1e-6, x_out=None, xo_bs=0, xo_rs=0, h=1024 * MB, h_bs=6400, h_rs=64)
GATED = dict(y=300 * MB, y_bs=6400, y_rs=64, x_out=400 * MB, xo_bs=6400, xo_rs=64)


def _norm(lib, **kw):
    a = dict(NORM, **kw)
    return lib.flux_modulated_norm(*[a[k] for k in NORM], None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses stay off a GPU")
@pytest.mark.parametrize("kw", [
    {}, dict(norm=1), dict(eps=0.0), GATED, dict(GATED, x_out=256 * MB),
    dict(GATED, x_out=256 * MB, stream_f32=1), dict(scale=500 * MB, shift=500 * MB + 128,
                                                    scale_bs=384, shift_bs=384),
    dict(x_out=1024 * MB, gate=1024 * MB),  # not looked at without y
])
def test_norm_accepts(lib, kw):
    assert _on_device(_norm(lib, **kw))


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(h=None), -1), (dict(GATED, x_out=None), -1),
    (dict(B=0), -2), (dict(S=0), -2), (dict(dim=0), -2), (dict(dim=60), -2), (dict(dim=16392), -2),
    (dict(norm=2), -2), (dict(eps=-1.0), -2), (dict(eps=float("nan")), -2),
    (dict(eps=float("inf")), -2), (dict(stream_f32=2), -2), (dict(vec_f32=-1), -2),
    (dict(x_rs=60), -2), (dict(h_rs=32), -2), (dict(h_bs=64), -2), (dict(GATED, xo_bs=0), -2),
    (dict(scale=500 * MB, scale_bs=-8), -2), (dict(shift=500 * MB, shift_bs=4), -2),
    (dict(x=256 * MB + 8), -4), (dict(h=1024 * MB + 8), -4), (dict(scale=500 * MB + 8), -4),
    (dict(GATED, y=300 * MB + 2), -4), (dict(GATED, gate=500 * MB + 4), -4),
    (dict(h=256 * MB), -9),                       # over x
    (dict(GATED, h=300 * MB), -9),                # over y
    (dict(GATED, h=400 * MB), -9),                # over x_out
    (dict(GATED, x_out=300 * MB), -9),            # over y
    (dict(GATED, x_out=256 * MB + 128), -9),      # over x, a row on
    (dict(scale=1024 * MB + 64), -9),
])
def test_norm_refuses(lib, kw, code):
    assert _norm(lib, **kw) == code


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.linear(x, torch.zeros(64, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        binding.modulated_norm(x)


def test_vector_helper_shapes():
    v = torch.zeros(3, 16)
    assert binding._vector("gate", v, 3, 16, v.dtype, -1)[1] == 16
    assert binding._vector("gate", v[0], 3, 16, v.dtype, -1)[1] == 0
    assert binding._vector("gate", v[:1], 3, 16, v.dtype, -1)[1] == 0
    assert binding._vector("gate", v[0].expand(3, 16), 3, 16, v.dtype, -1)[1] == 0
    for bad in (v[:2], v[:, :8], v.T, v[None], v[:, ::2]):
        with pytest.raises(ValueError):
            binding._vector("gate", bad, 3, 16, v.dtype, -1)
    with pytest.raises(ValueError, match="like the other vectors"):
        binding._vector("gate", v, 3, 16, torch.bfloat16, -1)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        binding._vector_type(torch.float64)
    assert binding._vector_type(torch.float32) == 1 and binding._vector_type(torch.bfloat16) == 0


def test_reference_linear_against_torch():
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    x, x2, w, b, gate, res = r(2, 5, 24), r(2, 5, 8), r(16, 32), r(16), r(2, 16), r(2, 5, 16)
    z = torch.nn.functional.linear(torch.cat([x, x2], -1).double(), w.double(), b.double())
    for act, f in (("silu", torch.nn.functional.silu), (None, lambda t: t),
                   ("gelu_tanh", lambda t: torch.nn.functional.gelu(t, approximate="tanh"))):
        want = res.double() + gate.double()[:, None] * f(z)
        got, bound = R.linear(x, w, x2, b, act, gate, res)
        assert (got - want).abs().max() < 1e-12
        R.check(want.bfloat16(), (got, bound), act)
    glu, _ = R.linear(x, w, x2, b, "swiglu")
    assert (glu - torch.nn.functional.silu(z[..., :8]) * z[..., 8:]).abs().max() < 1e-12


def test_reference_norm_against_torch():
    g = torch.Generator().manual_seed(6)
    x = (torch.randn(2, 5, 40, generator=g) * 3 + 2).bfloat16()
    y, gate, sc, sh = (torch.randn(*s, generator=g).bfloat16()
                       for s in ((2, 5, 40), (2, 40), (2, 40), (2, 40)))
    d = x.double() + gate.double()[:, None] * y.double()
    for kind, f in (("layer", lambda t: torch.nn.functional.layer_norm(t, (40,), eps=1e-6)),
                    ("rms", lambda t: torch.nn.functional.rms_norm(t, (40,), eps=1e-6))):
        want = f(d) * (1 + sc.double()[:, None]) + sh.double()[:, None]
        (h, hb), (xo, xb) = R.modulated_norm(x, sc, sh, y, gate, kind)
        assert (h - want).abs().max() < 1e-12 and (xo - d).abs().max() < 1e-12
        R.check(want.bfloat16(), (h, hb), kind)
        R.check(d.bfloat16(), (xo, xb), kind)


def test_bounds_catch_mistakes():
    """The bounds are tight enough: a lost channel, a bias taken twice, a norm
    without eps' place or with the biased mean left out break them."""
    g = torch.Generator().manual_seed(7)
    x, w = torch.randn(1, 9, 128, generator=g).bfloat16(), torch.randn(32, 128, generator=g).bfloat16()
    b = torch.randn(32, generator=g)
    ref = R.linear(x, w, bias=b)
    for bad in (R.linear(x[..., :127], w[:, :127], bias=b)[0], R.linear(x, w, bias=2 * b)[0],
                R.linear(x, w.roll(1, 0), bias=b)[0], R.linear(x, w, bias=b, act="silu")[0]):
        with pytest.raises(AssertionError):
            R.check(bad.bfloat16(), ref, "mistake")
    h, _ = R.modulated_norm(x + 1)
    for bad in (R.modulated_norm(x + 1, norm="rms")[0][0], R.modulated_norm(x + 1, eps=1e-1)[0][0],
                torch.nn.functional.layer_norm(x.double() + 1, (128,)) * (127 / 128) ** 2):
        with pytest.raises(AssertionError):
            R.check(bad.bfloat16(), h, "mistake")
