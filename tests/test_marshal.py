"""The compiled marshalling of the 8-bit products and the cross-attention: built and
in use, it makes the calls that the Python marshalling makes, and leaves to it
whatever it does not take."""
import pytest
import torch

from diffusion_transformer_joint_gb300 import binding, build


@pytest.fixture(scope="module")
def compiled():
    build.build()
    build.build_marshal()
    if binding._lib is not None and binding._compiled is None:
        binding._load_compiled(binding._lib)
    binding.load()
    return binding._compiled


def test_what_it_does_not_take(compiled):
    """CPU tensors, other objects, wrong numbers of arguments, tensors without memory:
    None, no exception."""
    x = torch.zeros(2, 4, 2, 128, dtype=torch.bfloat16)
    odd = (x, x.to("meta"), x.to_sparse(), 3, "x", None, object())
    for a in odd:
        for b in odd:
            assert compiled.quantize_fp8(a, 1, b, None) is None
            assert compiled.linear_fp8(a, b, a, b, None, None, None, None, None, None) is None
            assert compiled.cross_attention(a, b, b, None, None, None, None, None) is None
    assert compiled.quantize_fp8() is None
    assert compiled.linear_fp8(x) is None
    assert compiled.cross_attention(*[x] * 9) is None


@pytest.mark.gpu
def test_same_calls_as_in_python(compiled):
    """Every argument, given and left out: the library is called with the same
    values either way, but for the memory of outputs that the call makes."""
    g = torch.Generator().manual_seed(1)
    B, S, K, N = 3, 50, 400, 256
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, wide = r(B, S, K).bfloat16(), r(B, S + 4, 512).bfloat16()
    q, xs = binding.quantize_fp8(x)
    w, ws = binding.quantize_fp8(r(N, K), rows=128)
    res = r(B, S + 2, N).bfloat16()[:, 2:]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    h = wide.unflatten(-1, (4, 128))
    mask = (torch.rand(B, S + 4, generator=g) < 0.7).cuda()
    lengths = torch.tensor([5, 0, 54], dtype=torch.int32, device="cuda")
    calls = [
        (binding.quantize_fp8, (x,), {}), (binding.quantize_fp8, (x.float(),), {}),
        (binding.quantize_fp8, (x[0],), {}), (binding.quantize_fp8, (wide[:, 2:, 64:464],), {}),
        (binding.quantize_fp8, (r(300, 272),), dict(rows=128)),
        (binding.quantize_fp8, (x,), dict(out=torch.empty_like(q), scale=torch.empty_like(xs))),
        (binding.linear_fp8, (q, xs, w, ws), {}), (binding.linear_fp8, (q[1], xs[1], w, ws), {}),
        (binding.linear_fp8, (q, xs, w, ws), dict(act="swiglu", bias=r(N), gate=r(B, N // 2))),
        (binding.linear_fp8, (q, xs, w, ws), dict(act="silu", gate=r(1, N).bfloat16(),
                                                  residual=res, status=status)),
        (binding.linear_fp8, (q, xs, w, ws), dict(act="gelu_tanh", gate=r(N), residual=res,
                                                  out=torch.empty_like(res))),
        (binding.cross_attention, (h, h, h), {}),
        (binding.cross_attention, (h[:, 4:], h[:, :, :2], h[:, :, 2:]), dict(mask=mask, scale=0.2)),
        (binding.cross_attention, (h, h, h), dict(lengths=lengths, mask=mask.byte(), status=status,
                                                  out=torch.empty_like(h))),
    ]
    made = []
    real = binding._compiled

    class Watch:
        def __getattr__(self, name):
            def call(*a):
                made.append(getattr(real, name)(*a))
                return made[-1]
            return call

    binding.take_status()
    binding.linear_fp8(q, xs, w, ws)  # (the library's own status word is known from here on)
    for fn, args, kw in calls:
        given = {k for k in ("out", "scale") if isinstance(kw.get(k), torch.Tensor)}
        binding._compiled = Watch()
        try:
            fast = fn(*args, **kw)
        finally:
            binding._compiled = real
        assert made[-1] is not None, (fn.__name__, kw.keys())
        fast = tuple(t.clone() for t in (fast if isinstance(fast, tuple) else (fast,)))
        slow = fn(*args, stream=torch.cuda.current_stream(), **kw)
        slow = slow if isinstance(slow, tuple) else (slow,)
        for a, b in zip(fast, slow):
            assert a.shape == b.shape and a.dtype == b.dtype
            assert given or a.stride() == b.stride()
            assert torch.equal(a.float(), b.float()), (fn.__name__, kw.keys())
    assert int(status.item()) == 0 and binding.take_status() == 0
    x_out = torch.empty_like(q)
    assert binding.quantize_fp8(x, out=x_out)[0] is x_out


@pytest.mark.gpu
def test_refusals_come_from_python(compiled):
    x = torch.zeros(2, 4, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(binding.FluxError) as e:
        binding.quantize_fp8(x, out=x.view(torch.float8_e4m3fn)[..., :256])  # over x
    assert e.value.status == -9
    with pytest.raises(ValueError, match="torch.float8_e4m3fn"):
        binding.quantize_fp8(x, out=x)
    with pytest.raises(ValueError, match="current device|CUDA"):
        binding.quantize_fp8(x.cpu())
