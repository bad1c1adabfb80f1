"""The cross-attention part of a block in 8 bits, its operators run together as a
denoiser runs them; their streams, graphs, far strides and refusals.

x = x + gate * (cross_attention(q, k, v) Wo^T): the modulated norm, quantisation,
the query product; keys and values side by side from the encoder's states, once
for a prompt; attention over the padded prompts; quantisation and the output
product onto the stream. Every step's output is compared with the step's 64-bit
value from the GPU's own inputs of that step."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build
from tests import block_reference as R
from tests import cross_reference as X
from tests import fp8_reference as F

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _weight(g, *shape):
    return binding.quantize_fp8((torch.randn(*shape, generator=g) * shape[-1] ** -0.5).cuda(), rows=128)


class _Part:
    """The tensors and steps of the part, and what the steps leave."""

    def __init__(self, B, S, S_e, H, dim, seed):
        g = torch.Generator().manual_seed(seed)
        self.H, self.D = H, dim // H
        self.x0 = torch.randn(B, S, dim, generator=g).bfloat16().cuda()
        self.x = self.x0.clone()
        self.states = torch.randn(B, S_e, dim, generator=g).bfloat16().cuda()
        self.mods = (0.3 * torch.randn(B, 3, dim, generator=g)).bfloat16().cuda()
        self.lengths = torch.tensor([S_e, S_e // 3][:B], dtype=torch.int32, device="cuda")
        self.wq, self.wkv, self.wo = (_weight(g, n, dim) for n in (dim, 2 * dim, dim))
        self.bkv = (0.1 * torch.randn(2 * dim, generator=g)).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def prompt(self, **kw):
        self.e, self.es = binding.quantize_fp8(self.states, **kw)
        kv = binding.linear_fp8(self.e, self.es, *self.wkv, bias=self.bkv, status=self.status, **kw)
        self.kv = kv.unflatten(-1, (2, self.H, self.D))

    def steps(self, **kw):
        m = self.mods
        self.h = binding.modulated_norm(self.x, scale=m[:, 0], shift=m[:, 1], **kw)
        self.hq, self.hs = binding.quantize_fp8(self.h, **kw)
        self.q = binding.linear_fp8(self.hq, self.hs, *self.wq, status=self.status, **kw)
        self.o = binding.cross_attention(self.q.unflatten(-1, (self.H, self.D)), self.kv[:, :, 0],
                                         self.kv[:, :, 1], lengths=self.lengths, status=self.status,
                                         **kw)
        self.oq, self.os = binding.quantize_fp8(self.o.flatten(2), **kw)
        binding.linear_fp8(self.oq, self.os, *self.wo, gate=m[:, 2], residual=self.x, out=self.x,
                           status=self.status, **kw)


@pytest.mark.parametrize("B,S,S_e,H,dim", [(2, 700, 77, 4, 512), (2, 20, 300, 2, 256),
                                           (1, 1, 1, 4, 256)])
def test_cross_attention_part_of_a_block(B, S, S_e, H, dim):
    p = _Part(B, S, S_e, H, dim, 5)
    p.prompt()
    p.steps()
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    for x, q, s in ((p.states, p.e, p.es), (p.h, p.hq, p.hs), (p.o.flatten(2), p.oq, p.os)):
        wq, ws = F.quantize(x)
        assert torch.equal(q.cpu().float(), wq.float()) and torch.equal(s.cpu(), ws)
    R.check(p.kv.flatten(2), F.linear(p.e, p.es, *p.wkv, bias=p.bkv), "keys and values")
    R.check(p.h, R.modulated_norm(p.x0, p.mods[:, 0], p.mods[:, 1])[0], "norm")
    R.check(p.q, F.linear(p.hq, p.hs, *p.wq), "queries")
    R.check(p.o, X.cross(p.q.unflatten(-1, (H, p.D)), p.kv[:, :, 0], p.kv[:, :, 1], p.lengths),
            "attention")
    R.check(p.x, F.linear(p.oq, p.os, *p.wo, gate=p.mods[:, 2], residual=p.x0), "output product")


def test_the_part_in_one_graph():
    p = _Part(2, 300, 77, 4, 512, 6)
    p.prompt()
    p.steps()
    p.steps()
    want = p.x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.steps()
    for _ in range(3):
        p.x.copy_(p.x0)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.x, want)
    assert int(p.status.item()) == 0


def test_two_streams_at_once():
    """Two parts side by side, many times: each leaves what it leaves alone. (Clusters
    that split channels or keys, CTA pairs and single CTAs share the SMs.)"""
    parts = [_Part(2, 40, 900, 4, 512, 7), _Part(1, 600, 77, 8, 1024, 8)]
    want = []
    for p in parts:
        p.prompt()
        p.steps()
        torch.cuda.synchronize()
        want.append(p.x.clone())
    streams = [torch.cuda.Stream() for _ in parts]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(60):
        for p, s in zip(parts, streams):
            with torch.cuda.stream(s):
                p.x.copy_(p.x0)
            p.steps(stream=s)
        for p in parts:  # (their memory came from the streams that used it)
            del p.h, p.hq, p.hs, p.q, p.o, p.oq, p.os
    torch.cuda.synchronize()
    for p, w in zip(parts, want):
        assert torch.equal(p.x, w) and int(p.status.item()) == 0


def test_strides_past_32_bits():
    """Batch elements 2^32 elements and more apart: e4m3, bf16, scales and masks."""
    g = torch.Generator().manual_seed(11)
    far = (1 << 32) + 128
    B, S, K, N = 2, 5, 256, 136
    x = torch.randn(B, S, K, generator=g).bfloat16().cuda()
    bytes_ = torch.empty(far + S * K, dtype=torch.uint8, device="cuda")
    q = bytes_.view(E4M3).as_strided((B, S, K), (far, K, 1))
    binding.quantize_fp8(x, out=q)
    w, ws = _weight(g, N, K)
    wide = torch.zeros(far + S * N, dtype=torch.bfloat16, device="cuda")
    out = wide.as_strided((B, S, N), (far, N, 1))
    xq, xs = F.quantize(x)
    scales = torch.empty(far // 8 + S * 2, device="cuda").as_strided((B, S, 2), (far // 8, 2, 1))
    scales.copy_(xs)
    assert torch.equal(q.cpu().float(), xq.float())
    binding.linear_fp8(q, scales, w, ws, out=out)
    R.check(out, F.linear(q, scales, w, ws), "linear")
    del bytes_, q
    H, D, Sk = 1, 128, 200
    qq = torch.randn(B, S, H, D, generator=g).bfloat16().cuda()
    kv = torch.randn(2, B, Sk, H, D, generator=g).bfloat16().cuda()
    k = wide[:far + Sk * D].as_strided((B, Sk, H, D), (far, D, D, 1)) if wide.numel() >= far + Sk * D \
        else torch.empty(far + Sk * D, dtype=torch.bfloat16, device="cuda").as_strided(
            (B, Sk, H, D), (far, D, D, 1))
    k.copy_(kv[0])
    mask = torch.zeros(far + Sk, dtype=torch.bool, device="cuda").as_strided((B, Sk), (far, 1))
    mask.copy_((torch.rand(B, Sk, generator=g) < 0.5).cuda())
    for queries in (qq, qq.repeat(1, 300, 1, 1)):
        got = binding.cross_attention(queries, k, kv[1], mask=mask)
        R.check(got, X.cross(queries, k, kv[1], mask=mask), "cross")
    del k, mask, wide, out
    torch.cuda.empty_cache()


def test_own_status_word_and_allocated_outputs_on_a_given_stream():
    assert binding.take_status() == 0
    g = torch.Generator().manual_seed(13)
    x = torch.randn(3, 40, 256, generator=g).bfloat16().cuda()
    w, ws = _weight(g, 264, 256)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q, xs = binding.quantize_fp8(x, stream=s)
    y = binding.linear_fp8(q, xs, w, ws, stream=s)
    o = binding.cross_attention(x.unflatten(-1, (2, 128)), x.unflatten(-1, (2, 128)),
                                x.unflatten(-1, (2, 128)), stream=s)
    s.synchronize()
    assert binding.take_status(s) == 0
    R.check(y, F.linear(q, xs, w, ws), "linear")
    v = x.unflatten(-1, (2, 128))
    R.check(o, X.cross(v, v, v), "cross")


def test_binding_refusals():
    x = torch.zeros(2, 4, 256, dtype=torch.bfloat16, device="cuda")
    q, xs = binding.quantize_fp8(x)
    w, ws = binding.quantize_fp8(torch.zeros(256, 256, device="cuda"), rows=128)
    h = x.unflatten(-1, (2, 128))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for bad in (lambda: binding.quantize_fp8(x.half()), lambda: binding.quantize_fp8(x[0, 0]),
                lambda: binding.quantize_fp8(x, rows=128), lambda: binding.quantize_fp8(x, rows=64),
                lambda: binding.quantize_fp8(x, out=x), lambda: binding.quantize_fp8(x, scale=xs[..., :1]),
                lambda: binding.quantize_fp8(x, scale=xs.double()),
                lambda: binding.quantize_fp8(x.transpose(1, 2)),
                lambda: binding.quantize_fp8(x[..., :250]),
                lambda: binding.linear_fp8(x, xs, w, ws), lambda: binding.linear_fp8(q, xs, w[:, :128], ws),
                lambda: binding.linear_fp8(q, xs[:1], w, ws), lambda: binding.linear_fp8(q, xs, w, ws[:1]),
                lambda: binding.linear_fp8(q, xs, w, ws, act="relu"),
                lambda: binding.linear_fp8(q, xs, w[:128], ws[:1], act="swiglu"),  # halves of 64
                lambda: binding.linear_fp8(q, xs, w, ws, bias=torch.zeros(8, device="cuda")),
                lambda: binding.linear_fp8(q, xs, w, ws, residual=x.float()),
                lambda: binding.linear_fp8(q, xs, w, ws, status=i32(0).float()),
                lambda: binding.cross_attention(h, h[:1], h[:1]), lambda: binding.cross_attention(h, h, h[:, :2]),
                lambda: binding.cross_attention(h.float(), h, h), lambda: binding.cross_attention(h[0], h, h),
                lambda: binding.cross_attention(h, h, h, lengths=i32(4)),
                lambda: binding.cross_attention(h, h, h, lengths=i32(4, 4).long()),
                lambda: binding.cross_attention(h, h, h, mask=torch.ones(2, 4, device="cuda")),
                lambda: binding.cross_attention(h, h, h, mask=torch.ones(2, 5, dtype=torch.bool,
                                                                         device="cuda")),
                lambda: binding.cross_attention(h, h, h, scale=0.0),
                lambda: binding.cross_attention(h, h, h, scale=float("nan")),
                lambda: binding.cross_attention(h, h, h, out=h),
                lambda: binding.cross_attention(h.transpose(1, 2), h, h),
                lambda: binding.cross_attention(h[..., ::2], h[..., ::2], h[..., ::2])):
        with pytest.raises((ValueError, binding.FluxError)):
            bad()
    torch.cuda.synchronize()


def test_empty_prompts():
    """Lengths of zero for all: zeros, in both forms; the rows beside are left alone."""
    for Sq in (3, 2000):
        h = torch.full((2, Sq, 16, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(h, 7.0)
        binding.cross_attention(h, h[:, :3], h[:, :3], out=out,
                                lengths=torch.zeros(2, dtype=torch.int32, device="cuda"))
        assert bool((out == 0).all())
