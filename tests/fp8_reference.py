"""The products in 8-bit floating point written out, and how far the kernels may
be from them.

Quantisation is fp32 arithmetic rounded to nearest even at every step, so its
reference (the same steps in torch on the CPU) has to be met bit for bit.

The linear layer's reference takes the e4m3 values and the scales as exact.
A = sum |xs ws x w| over a row's channels. Bounds (u = 2^-24):

- e4m3 products have 8 significant bits, exact in fp32. The tensor core adds a
  group of 128 channels in four steps of 32; each aligns and truncates 33
  terms, twice those of a bf16 step of 16 channels, whose error is at most
  2^-22 of the sum of the magnitudes (tests/block_reference.py): 2^-21 of it a
  step, 2^-19 a group, and so 2^-19 A in all;
- the product of the two scales is off by u, the multiplication by it and the
  addition to the running sum by u each, of at most A; partial sums of up to
  eight ranges of channels are added: (G + 10) 2^-24 A with G groups.

E = 2^-19 A + (G + 10) 2^-24 A takes the place of the bf16 layer's E; what the
epilogue adds is as there.
"""
import math

import torch

from tests import block_reference as R

LEAST = 2.0 ** -100


def quantize(x, rows=1):
    """(e4m3 values, fp32 scales) of x [.., S, K] on the CPU, in fp32."""
    t = x.detach().float().cpu()
    lead, (S, K) = t.shape[:-2], t.shape[-2:]
    t = t.reshape(-1, S, K)
    sb, kb = -(-S // rows), -(-K // 128)
    a = torch.zeros(t.shape[0], sb * rows, kb * 128)
    a[:, :S, :K] = t.abs()
    top = a.reshape(-1, sb, rows, kb, 128).amax(dim=(2, 4)).clamp(min=LEAST)
    wide = top.repeat_interleave(rows, 1)[:, :S].repeat_interleave(128, 2)[:, :, :K]
    # (a number over a tensor would be its reciprocal's multiple, rounded twice)
    q = (t * (torch.tensor(448.0) / wide)).to(torch.float8_e4m3fn)
    return q.reshape(x.shape), (top / 448.0).reshape(*lead, sb, kb)


def values(q, scale, rows=1):
    """What e4m3 rows [.., S, K] and their scales stand for, in 64 bits on the CPU."""
    q, scale = q.detach().cpu().double(), scale.detach().cpu().double()
    S, K = q.shape[-2:]
    return q * scale.repeat_interleave(rows, -2)[..., :S, :].repeat_interleave(128, -1)[..., :K]


def linear(x, x_scale, w, w_scale, bias=None, act=None, gate=None, residual=None):
    """(reference, bound) in float64 on the CPU."""
    d = lambda t: t.detach().double().cpu()  # noqa: E731
    xd, wd = values(x, x_scale), values(w, w_scale, 128)
    y, A = xd @ wd.T, xd.abs() @ wd.abs().T
    if bias is not None:
        y, A = y + d(bias), A + d(bias).abs()
    E = (2.0 ** -19 + (-(-xd.shape[-1] // 128) + 10) * 2.0 ** -24) * A
    if act == "swiglu":
        n = y.shape[-1] // 2
        g, u, eg, eu = y[..., :n], y[..., n:], E[..., :n], E[..., n:]
        s = g * torch.sigmoid(g)
        out = s * u
        err = R.MAX_SLOPE * eg * (u.abs() + eu) + s.abs() * eu
        err = err + out.abs() * (8 + 1.2 * g.abs()) * 2.0 ** -23
    elif act == "silu":
        out = y * torch.sigmoid(y)
        err = R.MAX_SLOPE * E + out.abs() * (8 + 1.2 * y.abs()) * 2.0 ** -23
    elif act == "gelu_tanh":
        v = math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)
        out = 0.5 * y * (1 + torch.tanh(v))
        err = R.MAX_SLOPE * E + out.abs() * (8 + 2.4 * v.abs()) * 2.0 ** -23
    else:
        out, err = y, E
    if gate is not None:
        g = d(gate)
        g = g[:, None] if g.dim() == 2 else g
        out, err = out * g, err * g.abs()
    if residual is not None:
        out = out + d(residual)
        err = err + 2.0 ** -23 * out.abs()
    err = err + 2.0 ** -23 * out.abs()
    return out, err + R.BF16_HALF * (out.abs() + err) + 2.0 ** -133
