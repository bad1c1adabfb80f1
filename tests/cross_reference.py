"""Cross-attention written out in 64 bits, and how far the kernel may be from it.

Inputs are taken as exact. u = 2^-24 is half an fp32 step, h = 2^-8 half a bf16
step. Per row, with scores z_j = scale q . k_j, weights w_j = softmax_j(z):

- z_j: D products of 16 significant bits, exact, added by the tensor core in D/16
  steps, each off by at most 2^-22 of the sum of the magnitudes
  (tests/block_reference.py): dz = (D/16) 2^-22 scale sum |q||k_j|. Times log2(e)
  and less the maximum in one fused operation, and the base-2 exponential:
  2^-22 + |z_j - m| 2^-23 relative, with |z_j - m| <= 2 max |z|;
- so an unrounded weight p_j is off by e_j = dz_j + dz_max + (1 + 2 max |z|) 2^-22
  relative (the maximum cancels in p / l, its error does not enter twice, but is
  counted);
- the product with v takes p_j rounded to bf16, h more; l sums the unrounded
  ones in fp32, at most n_tiles + 40 additions deep, u each;
- sum_j p_j v_j is added by the tensor core in Sk/16 steps: (Sk/16) 2^-22 of the
  sum of the magnitudes; the parts' and streams' joining and the rescaling add
  2^-20;
- the output is rounded once to bf16.

All but the last are relative to A = sum_j w_j |v_j| per channel.
"""
import math

import torch


def cross(q, k, v, lengths=None, mask=None, scale=None):
    """(reference, bound), [B, Sq, H, D] in float64 on the CPU."""
    d = lambda t: t.detach().double().cpu()  # noqa: E731
    q, k, v = d(q), d(k), d(v)
    B, Sq, H, D = q.shape
    Sk, Hk = k.shape[1:3]
    scale = D ** -0.5 if scale is None else scale
    ref, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    for b in range(B):
        keep = torch.ones(Sk, dtype=torch.bool)
        if lengths is not None:
            keep &= torch.arange(Sk) < int(lengths[b])
        if mask is not None:
            keep &= mask[b].cpu() != 0
        if not keep.any():
            continue
        for h in range(H):
            kk, vv, qq = k[b, keep, h * Hk // H], v[b, keep, h * Hk // H], q[b, :, h]
            z = scale * qq @ kk.T
            dz = D / 16 * 2.0 ** -22 * scale * (qq.abs() @ kk.abs().T)
            w = torch.softmax(z, -1)
            top = z.abs().amax(-1, keepdim=True)
            e = dz + dz.amax(-1, keepdim=True) + (1 + 2 * top * math.log2(math.e)) * 2.0 ** -22
            e = e + 2.0 ** -8 + (Sk / 128 + 40) * 2.0 ** -24 + Sk / 16 * 2.0 ** -22 + 2.0 ** -20
            # the weights' errors also move l, by their weighted mean
            mean = (w * e).sum(-1, keepdim=True)
            r = w @ vv
            err = (w * e) @ vv.abs() + mean * (w @ vv.abs())
            ref[b, :, h] = r
            bound[b, :, h] = err + 2.0 ** -8 * (r.abs() + err) + 2.0 ** -133
    return ref, bound
