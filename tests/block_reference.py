"""The operators around the attention in a block, written out in 64 bits, and
how far a kernel with fp32 sums and one final rounding may be from them.

References take the bf16 / fp32 inputs as exact values. Bounds are derived,
per element, from the roundings of such a kernel (u = 2^-24, half an fp32
step):

- a tensor-core sum over K products in steps of 16: each of the K/16 steps
  aligns and truncates its 17 terms and the running sum, together at most
  2^-22 of the sum A of the magnitudes, and up to eight partial sums are added
  in fp32: |y - exact| <= (K/16 + 16) 2^-22 A =: E;
- the activation moves that by at most its slope (SiLU and GELU: below 1.13)
  and adds its own error: exp with argument v is off by at most
  (2 + 1.2 |v|) 2^-23, the division, the products and sums by u each:
  |act| (8 + 1.2 |v|) 2^-23;
- gate and residual add at most 2u each; the final bf16 rounding is half a
  step, 2^-8 of the value;
- the norm's mean and mean square are trees of at most 64 fp32 additions per
  thread and 10 more levels: relative 2^-17 of the mean magnitude; a
  difference v - mean is off by u (|v| + |mean|) and by the mean's error.
"""
import math

import torch

BF16_HALF = 2.0 ** -8
MAX_SLOPE = 1.13


def linear(x, w, x2=None, bias=None, act=None, gate=None, residual=None):
    """(reference, bound) of residual + gate * act([x | x2] W^T + bias), [B, S, N]
    in float64 on the CPU; gate [B, N] or [N]."""
    d = lambda t: t.detach().double().cpu()  # noqa: E731
    xs = d(x) if x2 is None else torch.cat([d(x), d(x2)], dim=-1)
    wd = d(w)
    y = xs @ wd.T
    mag = xs.abs() @ wd.abs().T
    if bias is not None:
        y, mag = y + d(bias), mag + d(bias).abs()
    E = (xs.shape[-1] / 16 + 16) * 2.0 ** -22 * mag
    if act == "swiglu":
        n = y.shape[-1] // 2
        g, u, eg, eu = y[..., :n], y[..., n:], E[..., :n], E[..., n:]
        s = g * torch.sigmoid(g)
        out = s * u
        err = MAX_SLOPE * eg * (u.abs() + eu) + s.abs() * eu
        err = err + out.abs() * (8 + 1.2 * g.abs()) * 2.0 ** -23
    elif act == "silu":
        out = y * torch.sigmoid(y)
        err = MAX_SLOPE * E + out.abs() * (8 + 1.2 * y.abs()) * 2.0 ** -23
    elif act == "gelu_tanh":
        v = math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)
        out = 0.5 * y * (1 + torch.tanh(v))
        err = MAX_SLOPE * E + out.abs() * (8 + 2.4 * v.abs()) * 2.0 ** -23
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
    return out, err + BF16_HALF * (out.abs() + err) + 2.0 ** -133


def modulated_norm(x, scale=None, shift=None, y=None, gate=None, norm="layer", eps=1e-6):
    """((h, bound), (x_out, bound)) in float64; x_out's bound is for its own type."""
    d = lambda t: t.detach().double().cpu()  # noqa: E731
    vec = lambda t: d(t)[:, None] if t.dim() == 2 else d(t)  # noqa: E731
    v = d(x)
    ev = torch.zeros_like(v)
    if y is not None:
        add = d(y) * (vec(gate) if gate is not None else 1.0)
        v = v + add
        ev = 2.0 ** -23 * (v.abs() + add.abs())
    half = BF16_HALF if x.dtype == torch.bfloat16 else 2.0 ** -24
    x_out = (v, ev + half * (v.abs() + ev) + 2.0 ** -133)
    if norm == "layer":
        m = v.mean(-1, keepdim=True)
        em = 2.0 ** -17 * v.abs().mean(-1, keepdim=True)
    else:
        m = em = torch.zeros_like(v[..., :1])
    c = v - m
    ec = ev + em + 2.0 ** -24 * (v.abs() + m.abs())
    ms = (c * c).mean(-1, keepdim=True)
    ems = (2 * c.abs() * ec + ec * ec).mean(-1, keepdim=True) + 2.0 ** -17 * ms
    r = 1 / torch.sqrt(ms + eps)
    er = 0.5 * r * ems / (ms + eps) + 2.0 ** -22 * r
    h = c * r
    eh = ec * (r + er) + c.abs() * er + 2.0 ** -23 * h.abs()
    if scale is not None:
        s = 1 + vec(scale)
        h, eh = h * s, eh * s.abs() + 2.0 ** -22 * (h * s).abs() + 2.0 ** -23 * h.abs()
    if shift is not None:
        h = h + vec(shift)
        eh = eh + 2.0 ** -23 * h.abs()
    return (h, eh + BF16_HALF * (h.abs() + eh) + 2.0 ** -133), x_out


def check(got, ref, what):
    """Every element of `got` within its bound of the reference."""
    want, bound = ref
    g = got.detach().double().cpu().reshape(want.shape)
    assert torch.isfinite(g).all(), what
    excess = (g - want).abs() - bound
    worst = int(excess.argmax())
    assert excess.flatten()[worst] <= 0, (
        f"{what}: element {worst} is {g.flatten()[worst]:.6g}, not {want.flatten()[worst]:.6g} "
        f"(bound {bound.flatten()[worst]:.3g})")
