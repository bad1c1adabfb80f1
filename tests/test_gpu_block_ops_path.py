"""The block operators run together, as the FLUX.2 blocks run them, against the
same steps in 64 bits with the tensors between calls rounded to bf16 as the
calls store them.

Blocks as in "Diffusers 中 Flux2Transformer2DModel 全面解析", section
内部架构双流块与单流块: modulation vectors from the activated timestep embedding;
modulated norm; products; joint attention; the output product gated onto the
residual; in the double-stream block a gated feed-forward with its own norm,
scale, shift and gate. Every step's GPU output is compared with the step's
64-bit value from the GPU's own inputs of that step, within the step's bound,
so that an error is seen where it is made.
"""
import numpy as np
import pytest
import torch

import oracle
from diffusion_transformer_joint_gb300 import binding, build
from diffusion_transformer_joint_gb300 import workloads as W
from tests import block_reference as R

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    binding.load()


def _weights(g, *shape):
    return (torch.randn(*shape, generator=g) * shape[-1] ** -0.5).bfloat16().cuda()


def _modulation(temb, w, dim, n):
    """The n modulation vectors [B, dim] of one product, checked."""
    mods = binding.linear(temb, w)
    R.check(mods, R.linear(temb, w), "modulation")
    return mods.reshape(temb.shape[0], n, dim).unbind(1)


def _attention(q, k, v, ids, S_t, norm):
    out = binding.joint_rope_attention(
        q, k, v, torch.from_numpy(ids[:S_t]).cuda(), torch.from_numpy(ids[S_t:]).cuda(),
        qk_norm=tuple(torch.from_numpy(n).cuda() for n in norm) + (EPS,))
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    ref = oracle.joint_rope_attention(f(q), f(k), f(v), ids[:S_t], ids[S_t:],
                                      qk_norm=tuple(norm) + (EPS,))
    # The attention's bar, max 1e-2 and mean 1e-3, is for v ~ N(0, 1) and logits of
    # standard deviation 1. An output is sum_j w_j v_j: a relative error of a
    # weight and a rounding of v move it in proportion to v, and a weight's
    # error is that of its logit, off by 2.1e-3 of the logits' deviation. So the
    # bar grows with the rms of v and with the largest product of a query and a
    # key norm weight (normalised rows: the logits' deviation is at most that).
    scale = max(1.0, float(np.sqrt((f(v) ** 2).mean())))
    scale *= max(1.0, max(norm[0].max(), norm[2].max()) * max(norm[1].max(), norm[3].max()))
    err = np.abs(f(out) - ref)
    assert err.max() <= 1e-2 * scale and err.mean() <= 1e-3 * scale
    return out


def test_timestep_embedding_and_single_stream_block():
    B, S_t, S_i, H, mlp = 2, 24, 100, 2, 768
    S, dim = S_t + S_i, H * 128
    g = torch.Generator().manual_seed(21)
    x = torch.randn(B, S, dim, generator=g).bfloat16().cuda()
    ids = W.random_ids(S, 22, 0, 100)
    norm = [np.random.default_rng(23 + i).uniform(0.5, 1.5, 128).astype(np.float32)
            for i in range(4)]
    sinusoids = torch.randn(B, 256, generator=g).bfloat16().cuda()
    w1, w2 = _weights(g, dim, 256), _weights(g, dim, dim)
    h = binding.linear(sinusoids, w1, act="silu")
    R.check(h, R.linear(sinusoids, w1, act="silu"), "timestep in")
    temb = binding.linear(h, w2, act="silu")
    R.check(temb, R.linear(h, w2, act="silu"), "timestep out")
    shift, scale, gate = _modulation(temb, _weights(g, 3 * dim, dim), dim, 3)

    h = binding.modulated_norm(x, scale=scale, shift=shift)
    R.check(h, R.modulated_norm(x, scale, shift)[0], "norm")
    w_in = _weights(g, 3 * dim + 2 * mlp, dim)
    q, k, v, act = binding.qkv_mlp_proj(h, w_in, H, mlp)
    for got, lo in ((q, 0), (k, dim), (v, 2 * dim)):
        R.check(got.reshape(B, S, dim), R.linear(h, w_in[lo:lo + dim]), "q, k, v")
    R.check(act, R.linear(h, w_in[3 * dim:], act="swiglu"), "mlp in")
    att = _attention(q, k, v, ids, S_t, norm).reshape(B, S, dim)
    w_out = _weights(g, dim, dim + mlp)
    ref = R.linear(att, w_out, x2=act, gate=gate, residual=x)
    out = binding.linear(att, w_out, x2=act, gate=gate, residual=x, out=x)
    assert out is x
    R.check(out, ref, "output product")


def test_double_stream_block_in_the_joint_layout():
    """Text and image streams live in one joint [B, S, dim] buffer; each has its
    own modulation and weights, and its rows are updated in place."""
    B, S_t, S_i, H = 2, 40, 300, 2
    S, dim = S_t + S_i, H * 128
    mlp = 3 * dim
    g = torch.Generator().manual_seed(31)
    joint = torch.randn(B, S, dim, generator=g).bfloat16().cuda()
    temb = torch.randn(B, dim, generator=g).bfloat16().cuda()
    ids = W.random_ids(S, 32, 0, 100)
    norm = [np.ones(128, np.float32) * (1 + 0.1 * i) for i in range(4)]
    rows = {"text": slice(0, S_t), "image": slice(S_t, S)}
    mods = {s: _modulation(temb, _weights(g, 6 * dim, dim), dim, 6) for s in rows}
    qkv = torch.empty(3, B, S, H, 128, dtype=torch.bfloat16, device="cuda")
    h = torch.empty_like(joint)
    for s, r in rows.items():
        shift, scale = mods[s][:2]
        binding.modulated_norm(joint[:, r], scale=scale, shift=shift, out=h[:, r])
        R.check(h[:, r], R.modulated_norm(joint[:, r], scale, shift)[0], f"{s} norm")
        for i in range(3):  # to_q, to_k, to_v with bias, straight into the joint layout
            w, b = _weights(g, dim, dim), (0.1 * torch.randn(dim, generator=g)).cuda()
            out = qkv[i].reshape(B, S, dim)[:, r]
            binding.linear(h[:, r], w, bias=b, out=out)
            R.check(out, R.linear(h[:, r], w, bias=b), f"{s} qkv {i}")
    att = _attention(*qkv, ids, S_t, norm).reshape(B, S, dim)
    for s, r in rows.items():
        gate, shift, scale, gate2 = mods[s][2:]
        w = _weights(g, dim, dim)
        ref = R.linear(att[:, r], w, gate=gate, residual=joint[:, r])
        binding.linear(att[:, r], w, gate=gate, residual=joint[:, r], out=joint[:, r])
        R.check(joint[:, r], ref, f"{s} attention out")
        n = binding.modulated_norm(joint[:, r], scale=scale, shift=shift)
        R.check(n, R.modulated_norm(joint[:, r], scale, shift)[0], f"{s} second norm")
        w1, w2 = _weights(g, 2 * mlp, dim), _weights(g, dim, mlp)
        ff = binding.linear(n, w1, act="swiglu")
        R.check(ff, R.linear(n, w1, act="swiglu"), f"{s} feed-forward in")
        ref = R.linear(ff, w2, gate=gate2, residual=joint[:, r])
        binding.linear(ff, w2, gate=gate2, residual=joint[:, r], out=joint[:, r])
        R.check(joint[:, r], ref, f"{s} feed-forward out")


def test_tensor_parallel_output_product():
    """Two ranks' calls, one after the other on one GPU: each multiplies its
    heads' columns of the output weight in place; the summed product meets the
    fp32 residual stream in the next block's norm."""
    B, S, H, dim = 1, 150, 4, 512
    g = torch.Generator().manual_seed(41)
    att = torch.randn(B, S, H * 128, generator=g).bfloat16().cuda()
    w = _weights(g, dim, H * 128)
    parts = []
    for lo in (0, H * 64):
        cols = slice(lo, lo + H * 64)
        parts.append(binding.linear(att[..., cols], w[:, cols]))
        R.check(parts[-1], R.linear(att[..., cols], w[:, cols]), "rank's part")
    y = (parts[0].float() + parts[1].float()).bfloat16()  # the all-reduce
    x = torch.randn(B, S, dim, generator=g).cuda()
    mods = torch.randn(B, 3, dim, generator=g).cuda()
    ref, ref_x = R.modulated_norm(x, mods[:, 0], mods[:, 1], y, mods[:, 2])
    h, x2 = binding.modulated_norm(x, scale=mods[:, 0], shift=mods[:, 1], y=y, gate=mods[:, 2],
                                   x_out=x)
    assert x2 is x
    R.check(h, ref, "norm")
    R.check(x, ref_x, "residual stream")


def test_block_in_one_graph():
    """Norm, product, norm and product captured together replay as run eagerly."""
    B, S, dim = 1, 333, 256
    g = torch.Generator().manual_seed(51)
    x = torch.randn(B, S, dim, generator=g).bfloat16().cuda()
    m = (0.3 * torch.randn(B, 6, dim, generator=g)).bfloat16().cuda()
    w1, w2 = _weights(g, 6 * dim, dim), _weights(g, dim, 3 * dim)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, f = torch.empty_like(x), torch.empty(B, S, 3 * dim, dtype=torch.bfloat16, device="cuda")
    stream = x.clone()

    def steps():
        binding.modulated_norm(stream, scale=m[:, 0], shift=m[:, 1], out=h)
        binding.linear(h, w1, act="swiglu", out=f, status=status)
        binding.linear(f, w2, gate=m[:, 2], residual=stream, out=stream, status=status)

    steps()
    steps()
    want = stream.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(3):
        stream.copy_(x)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(stream, want)
    assert int(status.item()) == 0
