"""Calls that the Python marshalling refuses are not made by the compiled one either:
the same exception with the same words, whichever of the two a call begins in."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def t():
    build.build()
    build.build_marshal()
    binding.load()
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, xs = binding.quantize_fp8(r(2, 20, 256))
    w, ws = binding.quantize_fp8(r(256, 256), rows=128)
    h = r(2, 20, 4, 64).bfloat16()
    return dict(raw=r(2, 20, 256).bfloat16(), x=x, xs=xs, w=w, ws=ws, h=h, r=r)


Q, L, X = binding.quantize_fp8, binding.linear_fp8, binding.cross_attention
LIN = ("x", "xs", "w", "ws")
CALLS = [
    (Q, lambda t: ((t["raw"],), dict(rows=2))),
    (Q, lambda t: ((t["raw"],), dict(rows=128))),
    (Q, lambda t: ((t["raw"],), dict(rows=0))),
    (Q, lambda t: ((t["raw"].half(),), {})),
    (Q, lambda t: ((t["raw"][0, 0],), {})),
    (Q, lambda t: ((t["raw"][..., ::2],), {})),
    (Q, lambda t: ((t["raw"][..., :250],), {})),
    (Q, lambda t: ((t["raw"][..., 4:244],), {})),
    (Q, lambda t: ((t["raw"],), dict(out=t["x"][:1]))),
    (Q, lambda t: ((t["raw"],), dict(out=t["raw"]))),
    (Q, lambda t: ((t["raw"],), dict(scale=t["xs"][..., :1]))),
    (Q, lambda t: ((t["raw"],), dict(scale=t["xs"].double()))),
    (Q, lambda t: ((t["raw"],), dict(scale=t["xs"][:, :1].expand(2, 20, 2)))),
    (Q, lambda t: ((t["raw"][:0],), {})),
    (Q, lambda t: ((t["raw"][:, :0],), {})),
    (L, lambda t: ((t["raw"], t["xs"], t["w"], t["ws"]), {})),
    (L, lambda t: ((t["x"], t["xs"][:1], t["w"], t["ws"]), {})),
    (L, lambda t: ((t["x"], t["xs"].half(), t["w"], t["ws"]), {})),
    (L, lambda t: ((t["x"], t["xs"].cpu(), t["w"], t["ws"]), {})),
    (L, lambda t: ((t["x"], t["xs"], t["w"][:, :128], t["ws"]), {})),
    (L, lambda t: ((t["x"], t["xs"], t["w"], t["ws"][:1]), {})),
    (L, lambda t: ((t["x"], t["xs"], t["w"][:200], t["ws"]), dict(act="swiglu"))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(act="relu"))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(bias=t["r"](255)))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(bias=t["r"](512)[::2]))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(bias=t["r"](256).half()))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(bias=t["r"](256), gate=t["r"](256).bfloat16()))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(gate=t["r"](3, 256)))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(gate=t["r"](2, 256).cpu()))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(gate=t["r"](2, 1, 256)))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(residual=t["raw"].float()))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(residual=t["raw"][0]))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(out=t["raw"][..., :128]))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(status=torch.zeros(1, device="cuda")))),
    (L, lambda t: (tuple(t[n] for n in LIN), dict(status=torch.zeros(1, dtype=torch.int32)))),
    (X, lambda t: ((t["h"][0], t["h"], t["h"]), {})),
    (X, lambda t: ((t["h"], t["h"].float(), t["h"]), {})),
    (X, lambda t: ((t["h"], t["h"], t["h"][:, 1:]), {})),
    (X, lambda t: ((t["h"], t["h"], t["h"][:, :, :2]), {})),
    (X, lambda t: ((t["h"], t["h"][:, :, :3], t["h"][:, :, :3]), {})),
    (X, lambda t: ((t["h"][..., :32], t["h"][..., :32], t["h"][..., :32]), {})),
    (X, lambda t: ((t["h"].transpose(1, 2), t["h"], t["h"]), {})),
    (X, lambda t: ((t["h"][:, :, ::2], t["h"], t["h"]), {})),
    (X, lambda t: ((t["h"][:1].expand(2, 20, 4, 64), t["h"], t["h"]), {})),
    (X, lambda t: ((t["h"], t["h"][:, :0], t["h"][:, :0]), {})),
    (X, lambda t: ((t["h"],) * 3, dict(lengths=torch.ones(2, dtype=torch.int64, device="cuda")))),
    (X, lambda t: ((t["h"],) * 3, dict(lengths=torch.ones(2, dtype=torch.int32)))),
    (X, lambda t: ((t["h"],) * 3, dict(lengths=torch.ones(4, dtype=torch.int32, device="cuda")[::2]))),
    (X, lambda t: ((t["h"],) * 3, dict(mask=torch.ones(2, 19, dtype=torch.bool, device="cuda")))),
    (X, lambda t: ((t["h"],) * 3, dict(mask=torch.ones(2, 20, device="cuda")))),
    (X, lambda t: ((t["h"],) * 3, dict(mask=torch.ones(20, 2, dtype=torch.bool, device="cuda").T))),
    (X, lambda t: ((t["h"],) * 3, dict(scale=0.0))),
    (X, lambda t: ((t["h"],) * 3, dict(scale=float("inf")))),
    (X, lambda t: ((t["h"],) * 3, dict(out=t["h"]))),
    (X, lambda t: ((t["h"],) * 3, dict(out=t["h"].clone()[:, :, :2]))),
    (X, lambda t: ((t["h"],) * 3, dict(status=torch.zeros(0, dtype=torch.int32, device="cuda")))),
]


@pytest.mark.parametrize("i", range(len(CALLS)))
def test_refused_alike(t, i):
    fn, make = CALLS[i]
    args, kw = make(t)
    said = []
    for stream in ({}, dict(stream=torch.cuda.current_stream())):
        with pytest.raises((ValueError, binding.FluxError)) as e:
            fn(*args, **kw, **stream)
        said.append((type(e.value), str(e.value)))
    assert said[0] == said[1]
