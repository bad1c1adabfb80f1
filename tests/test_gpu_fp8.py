"""binding.quantize_fp8 bit for bit, and binding.linear_fp8 against the 64-bit
definition: few and many rows, every epilogue, odd sizes, strided views."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R
from tests import fp8_reference as F

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _same(got, want, what):
    """Equal values, NaN where NaN is wanted."""
    got, want = got.detach().cpu().float(), want.float()
    assert got.shape == want.shape, what
    assert bool(((got == want) | (got.isnan() & want.isnan())).all()), what


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,S,K,rows", [
    (1, 1, 16, 1), (1, 1, 128, 1), (1, 3, 144, 1), (2, 77, 4096, 1), (3, 33, 400, 1),
    (1, 5000, 1040, 1), (2, 1, 96, 1),
    (1, 1, 16, 128), (1, 128, 128, 128), (1, 129, 144, 128), (1, 700, 1040, 128)])
def test_quantize(B, S, K, rows, dtype):
    g = torch.Generator().manual_seed(S + K)
    x = (torch.randn(B, S, K, generator=g) * torch.exp(3 * torch.randn(B, S, 1, generator=g)))
    x = x.to(dtype)[0] if rows > 1 else x.to(dtype)
    q, scale = binding.quantize_fp8(x.cuda(), rows=rows)
    assert q.dtype == E4M3 and scale.dtype == torch.float32
    wq, ws = F.quantize(x, rows)
    _same(scale, ws, "scales")
    _same(q, wq, "values")


def test_quantize_special_values():
    """Groups of zeros, tiny and huge values, infinities and NaN; each leaves the
    groups beside it as they are."""
    x = torch.ones(6, 384)
    x[0, 128:256] = 0.0
    x[1, 128:256] = 2.0 ** -126
    x[1, 130] = -(2.0 ** -110)
    x[2, 128:256] = 3e38
    x[3, 200] = float("inf")
    x[4, 255] = float("nan")
    x[5, 128:256] = 2.0 ** -140  # denormal
    for dtype in (torch.float32, torch.bfloat16):
        q, scale = binding.quantize_fp8(x.to(dtype).cuda())
        wq, ws = F.quantize(x.to(dtype))
        _same(scale, ws, dtype)
        _same(q, wq, dtype)
        v = F.values(q, scale)
        assert v[3, 128:256].isnan().all() and v[4, 128:256].isnan().all()
        assert torch.isfinite(v[[0, 1, 2, 5]]).all() and bool((v[0, 128:256] == 0).all())


def test_quantize_views_and_given_outputs():
    g = torch.Generator().manual_seed(3)
    buf = torch.randn(2, 50, 320, generator=g).bfloat16().cuda()
    x = buf[:, 7:, 16:288]
    qbuf = torch.zeros(2, 60, 512, dtype=torch.uint8, device="cuda").view(E4M3)
    out = qbuf[:, 3:46, 32:304]
    sbuf = torch.full((2, 3, 50), -1.0, device="cuda")
    scale = sbuf[:, :, :43].transpose(1, 2)
    q, s = binding.quantize_fp8(x, out=out, scale=scale)
    assert q is out and s is scale
    wq, ws = F.quantize(x)
    _same(q, wq, "values")
    _same(s, ws, "scales")
    assert bool((sbuf[:, :, 43:] == -1).all())
    rest = qbuf.view(torch.uint8).clone()
    rest[:, 3:46, 32:304] = 0
    assert int(rest.sum()) == 0
    rows_first = torch.empty(2, 43, 3, device="cuda")  # groups beside one another
    _same(binding.quantize_fp8(x, scale=rows_first)[1], ws, "scales")


def _make(B, S, K, N, act=None, bias=False, gate=False, residual=False, vec=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(1000 + seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rows = 2 * N if act == "swiglu" else N
    x, xs = F.quantize(r(B, S, K) * torch.exp(r(B, S, 1)))
    w, ws = F.quantize(r(rows, K) * K ** -0.5 * torch.exp(r(rows, 1)), 128)
    ops = dict(x=x, x_scale=xs, w=w, w_scale=ws, act=act)
    ops["bias"] = r(rows).to(vec) if bias else None
    ops["gate"] = r(B, N).to(vec) if gate else None
    ops["residual"] = (2 * r(B, S, N)).bfloat16() if residual else None
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in ops.items()}


def _run(ops, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = binding.linear_fp8(status=status, **ops, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out


FULL = dict(bias=True, gate=True, residual=True)


@pytest.mark.parametrize("B,S,K,N,kw", [
    (1, 1, 16, 8, {}),                                     # the smallest call
    (1, 1, 256, 1024, dict(act="silu")),
    (1, 1, 4096, 128, FULL),                               # channels over eight CTAs
    (2, 1, 512, 384, dict(bias=True)),                     # batch elements joined
    (1, 2, 144, 40, dict(FULL, act="gelu_tanh")),          # ragged channels and features
    (1, 17, 2048, 248, FULL),
    (1, 9, 1008, 256, dict(act="swiglu", bias=True)),
    (3, 5, 272, 128, dict(FULL, act="swiglu")),
    (1, 64, 640, 136, dict(residual=True)),
    (1, 77, 768, 640, dict(FULL, act="swiglu", vec=torch.float32)),
    (2, 77, 4096, 1024, dict(FULL, vec=torch.float32)),
    (1, 130, 400, 520, dict(FULL, act="silu")),
    (1, 256, 128, 1032, {}),
])
def test_few_rows(B, S, K, N, kw):
    ops = _make(B, S, K, N, **kw)
    R.check(_run(ops), F.linear(**ops), f"{B}x{S}x{K}->{N}")


@pytest.mark.parametrize("B,S,K,N,kw", [
    (1, 300, 208, 136, FULL),
    (1, 513, 80, 520, dict(FULL, act="gelu_tanh")),
    (1, 1100, 512, 2048, dict(FULL, vec=torch.float32)),
    (2, 700, 528, 1544, dict(FULL, vec=torch.float32)),     # a gate per batch element, joined
    (3, 390, 256, 1280, dict(FULL, act="swiglu")),
    (1, 2500, 2064, 768, dict(act="swiglu", vec=torch.float32, bias=True)),
    (1, 3000, 144, 4104, dict(gate=True, residual=True)),   # more tiles than pairs
    (1, 4056, 1024, 1000, dict(bias=True, act="silu")),
    (1, 2600, 16, 4096, dict(residual=True)),
])
def test_many_rows(B, S, K, N, kw):
    ops = _make(B, S, K, N, **kw)
    R.check(_run(ops), F.linear(**ops), f"{B}x{S}x{K}->{N}")


@pytest.mark.parametrize("B,S,K,N", [(2, 21, 272, 72), (3, 1, 144, 72), (2, 600, 272, 1032)])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_views(B, S, K, N, act):
    """Operands and output inside wider buffers, scales in other orders; what lies
    around the output is left as it was."""
    N = 128 * (N // 72) if act else N
    ops = _make(B, S, K, N, act=act, **FULL, seed=S)
    out_buf = torch.full((B, S + 7, N + 48), 7.0, dtype=torch.bfloat16, device="cuda")
    xbuf = torch.full((B, S + 5, K + 48), 0x7F, dtype=torch.uint8, device="cuda").view(E4M3)
    xbuf[:, 5:, 16:16 + K] = ops["x"]
    wbuf = torch.full((ops["w"].shape[0], K + 80), 0x7F, dtype=torch.uint8,
                      device="cuda").view(E4M3)
    wbuf[:, 64:64 + K] = ops["w"]
    rbuf = torch.full((B, S + 1, N + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    rbuf[:, 1:, 8:8 + N] = ops["residual"]
    ops.update(x=xbuf[:, 5:, 16:16 + K], w=wbuf[:, 64:64 + K], residual=rbuf[:, 1:, 8:8 + N])
    ops["x_scale"] = ops["x_scale"].permute(2, 0, 1).contiguous().permute(1, 2, 0)
    ops["w_scale"] = ops["w_scale"].T.contiguous().T
    out = out_buf[:, 7:, 16:16 + N]
    assert _run(ops, out=out) is out
    R.check(out, F.linear(**ops), "views")
    assert bool((out_buf[:, :7] == 7).all())
    assert bool((out_buf[:, 7:, :16] == 7).all() and (out_buf[:, 7:, 16 + N:] == 7).all())


@pytest.mark.parametrize("S", [1, 19, 1100])
def test_residual_in_place_and_one_scale_for_all(S):
    ops = _make(2, S, 256, 1032, **FULL, seed=S)
    ops["x_scale"] = torch.full((1, 1, 1), 0.25, device="cuda").expand(2, S, 2)
    ops["w_scale"] = torch.full((1, 1), 0.02, device="cuda").expand(9, 2)
    ref = F.linear(**ops)
    assert _run(ops, out=ops["residual"]) is ops["residual"]
    R.check(ops["residual"], ref, "in place")


@pytest.mark.parametrize("S,N", [(3, 520), (1500, 1032)])
def test_the_same_call_gives_the_same_bits(S, N):
    ops = _make(1, S, 1040, N, **FULL)
    a, b = _run(ops), _run(ops)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
