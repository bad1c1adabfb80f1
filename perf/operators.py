"""Cases for measuring the operators around the joint attention of a FLUX.2 block.

Two operators, each in a plain form (elementary torch operations in fp32, one
rounding at the end) and, with ``own`` set, as a user calls them:

- ``linear``: out = residual + gate * act([x | x2] W^T + bias), the products of
  a block that the fused input projection does not cover: the output
  projections, the feed-forward layers, the timestep MLP, the modulation
  layers and the final projection.
- ``norm``: x_out = x + gate * y, h = norm(x_out) * (1 + scale) + shift, the
  modulated norm before a block's products, fused with the gated residual of
  the product before it.

Shapes follow the workloads of this repository (hidden widths 4096 and 6144,
MLP width three times that, 512 text tokens, 4096 image tokens, 12800 tokens in
the two-reference edit).
"""
import math

import torch

own = False

BF16, F32 = "bfloat16", "float32"
EPS = 1e-6


def _linear(name, B, S, K, N, K2=0, act="none", bias=False, gate=False, residual=False, vec=BF16,
            strided=False):
    return {"op": "linear", "name": name, "B": B, "S": S, "K": K, "K2": K2, "N": N, "act": act,
            "bias": bias, "gate": gate, "residual": residual, "vec": vec, "strided": strided}


def _norm(name, B, S, dim, kind="layer", y=False, modulated=True, x=BF16, vec=BF16, strided=False):
    return {"op": "norm", "name": name, "B": B, "S": S, "dim": dim, "kind": kind, "y": y,
            "modulated": modulated, "x": x, "vec": vec, "strided": strided}


def listed():
    return [
        # first layer of the timestep MLP: one row of 256 sinusoids, once a step
        _linear("time_embed", 1, 1, 256, 4096, act="silu"),
        # a block's six modulation vectors for a guided pair: two rows over a wide weight
        _linear("modulation", 2, 1, 4096, 24576, bias=True),
        # the text stream's feed-forward out, two prompts of 77 tokens, in the joint layout
        _linear("text_ff_out", 2, 77, 12288, 4096, gate=True, residual=True, vec=F32,
                strided=True),
        # the text stream's gated feed-forward in, a full prompt
        _linear("text_ff_in", 1, 512, 4096, 12288, act="swiglu"),
        # the last layer: the image tokens (a 52 x 78 grid) to 128 latent channels
        _linear("final_proj", 1, 4056, 4096, 128, bias=True),
        # the image stream's attention output, gated onto the residual
        _linear("image_attn_out", 1, 4096, 4096, 4096, gate=True, residual=True),
        # the single-stream block's output product over [attention | MLP]
        _linear("single_out", 1, 4608, 4096, 4096, K2=12288, gate=True, residual=True),
        # the same at the widest model and the two-reference edit
        _linear("edit_single_out", 1, 12800, 6144, 6144, K2=18432, gate=True, residual=True),
        # one token
        _norm("one_token", 1, 1, 4096),
        # the image stream before its attention
        _norm("image_norm", 1, 4096, 4096),
        # a guided pair between two blocks: fp32 residual stream, the product's gated output added
        _norm("pair_gated", 2, 4608, 4096, y=True, x=F32, vec=F32),
        # the widest model's edit sequence between two blocks
        _norm("edit_gated", 1, 12800, 6144, y=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_FLOPS = 2.0 * 12800 * (6144 + 18432) * 6144
MOST_BYTES = 4.0 * 12800 * 6144 * 2


def draw(rng):
    """Sizes over the ranges of the listed cases, no costlier than the largest of them."""
    while True:
        if rng.random() < 0.6:
            c = _linear("", rng.choice((1, 1, 2, 3)), _log(rng, 1, 12800), 8 * _log(rng, 8, 2048),
                        8 * _log(rng, 8, 2048), act=rng.choice(("none", "none", "silu",
                                                                "gelu_tanh", "swiglu")),
                        bias=rng.random() < 0.5, gate=rng.random() < 0.5,
                        residual=rng.random() < 0.5, vec=rng.choice((BF16, F32)),
                        strided=rng.random() < 0.4)
            if rng.random() < 0.3:
                c["K2"] = 8 * _log(rng, 8, 2048)
        else:
            c = _norm("", rng.choice((1, 1, 2, 3)), _log(rng, 1, 12800), 8 * _log(rng, 8, 1024),
                      kind=rng.choice(("layer", "layer", "rms")), y=rng.random() < 0.5,
                      modulated=rng.random() < 0.8, x=rng.choice((BF16, BF16, F32)),
                      vec=rng.choice((BF16, F32)), strided=rng.random() < 0.4)
        w = work(c)
        if w["flops"] <= MOST_FLOPS and w["bytes"] <= MOST_BYTES:
            del c["name"]
            return c


def work(c):
    """Bytes read and written once, and the operations of the product or the norm."""
    rows = c["B"] * c["S"]
    if c["op"] == "linear":
        K, N = c["K"] + c["K2"], c["N"]
        wr = 2 * N if c["act"] == "swiglu" else N
        vb = 2 if c["vec"] == BF16 else 4
        b = 2 * (rows * K + wr * K + rows * N * (2 if c["residual"] else 1))
        b += vb * ((wr if c["bias"] else 0) + (c["B"] * N if c["gate"] else 0))
        return {"bytes": b, "flops": 2 * rows * wr * K}
    n, xb = rows * c["dim"], 2 if c["x"] == BF16 else 4
    vb = 2 if c["vec"] == BF16 else 4
    b = n * (xb + 2 + ((2 + xb) if c["y"] else 0))
    b += vb * c["B"] * c["dim"] * ((2 if c["modulated"] else 0) + (1 if c["y"] else 0))
    return {"bytes": b, "flops": n * (8 + (2 if c["y"] else 0))}


def _rows(c, g, width, dtype, scale=None, offset=0.0):
    """[B, S, width] rows; the trailing rows of a longer joint buffer when strided."""
    pad = 24 if c["strided"] else 0
    t = torch.randn((c["B"], pad + c["S"], width), generator=g, device="cuda")
    if scale is not None:
        t *= scale
    if offset:
        t += offset * torch.randn((c["B"], pad + c["S"], 1), generator=g, device="cuda")
    return t.to(dtype)[:, pad:]


def _channels(g, width):
    """Channel magnitudes as a network's activations have them: a few are several times the rest."""
    return torch.exp(0.6 * torch.randn(width, generator=g, device="cuda"))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    vec = getattr(torch, c["vec"])
    s = {"case": dict(c)}
    if c["op"] == "linear":
        K, K2, N = c["K"], c["K2"], c["N"]
        wr = 2 * N if c["act"] == "swiglu" else N
        s["x"] = _rows(c, g, K, torch.bfloat16, _channels(g, K))
        s["x2"] = _rows(c, g, K2, torch.bfloat16, _channels(g, K2)) if K2 else None
        w = torch.randn((wr, K + K2), generator=g, device="cuda")
        s["w"] = (w * (K + K2) ** -0.5).to(torch.bfloat16)
        s["bias"] = (0.2 * torch.randn(wr, generator=g, device="cuda")).to(vec) if c["bias"] else None
        s["gate"] = (0.5 * torch.randn((c["B"], N), generator=g, device="cuda")).to(vec) \
            if c["gate"] else None
        s["residual"] = _rows(c, g, N, torch.bfloat16, _channels(g, N)) if c["residual"] else None
        s["out"] = _rows(c, g, N, torch.bfloat16)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    dim, xt = c["dim"], getattr(torch, c["x"])
    s["x"] = _rows(c, g, dim, xt, _channels(g, dim), 0.5)
    s["y"] = _rows(c, g, dim, torch.bfloat16, _channels(g, dim)) if c["y"] else None
    mods = 0.3 * torch.randn((c["B"], 3, dim), generator=g, device="cuda")
    mods = mods.to(vec)  # the modulation layer's output: shift, scale, gate side by side
    s["shift"], s["scale"] = (mods[:, 0], mods[:, 1]) if c["modulated"] else (None, None)
    s["gate"] = mods[:, 2] if c["y"] else None
    s["h"] = _rows(c, g, dim, torch.bfloat16)
    s["x_out"] = _rows(c, g, dim, xt) if c["y"] else None
    return s


def _run_own(s):
    from diffusion_transformer_joint_gb300 import binding

    c = s["case"]
    if c["op"] == "linear":
        return binding.linear(s["x"], s["w"], x2=s["x2"], bias=s["bias"],
                              act=None if c["act"] == "none" else c["act"], gate=s["gate"],
                              residual=s["residual"], out=s["out"], status=s["status"])
    return binding.modulated_norm(s["x"], scale=s["scale"], shift=s["shift"], y=s["y"],
                                  gate=s["gate"], norm=c["kind"], eps=EPS, out=s["h"],
                                  x_out=s["x_out"])


def _plain_linear(s):
    c = s["case"]
    x = s["x"].float()
    if s["x2"] is not None:
        x = torch.cat([x, s["x2"].float()], dim=-1)
    y = x @ s["w"].float().T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["act"] == "swiglu":
        a, b = y[..., :c["N"]], y[..., c["N"]:]
        y = a / (1.0 + torch.exp(-a)) * b
    elif c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif c["act"] == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["gate"] is not None:
        y = y * s["gate"].float()[:, None]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    if s["y"] is not None:
        x = x + s["gate"].float()[:, None] * s["y"].float()
    d = x - x.mean(dim=-1, keepdim=True) if c["kind"] == "layer" else x
    h = d / torch.sqrt((d * d).mean(dim=-1, keepdim=True) + EPS)
    if s["scale"] is not None:
        h = h * (1.0 + s["scale"].float()[:, None]) + s["shift"].float()[:, None]
    h = h.to(torch.bfloat16)
    return h if s["y"] is None else (h, x.to(s["x"].dtype))


def run(state):
    if own:
        return _run_own(state)
    return _plain_linear(state) if state["case"]["op"] == "linear" else _plain_norm(state)


def exact(case, seed):
    """The definitions in 64 bits, the rows in pieces."""
    s = prepare(case, seed)
    c = s["case"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and
         k in ("w", "bias", "gate", "scale", "shift")}
    one = torch.ones((), dtype=torch.float64, device="cuda")
    parts = []
    for b in range(c["B"]):
        for lo in range(0, c["S"], 1024):
            r = slice(lo, min(lo + 1024, c["S"]))
            x = s["x"][b, r].double()
            if c["op"] == "linear":
                z = torch.einsum("mk,nk->mn", x, d["w"][:, :c["K"]])
                if c["K2"]:
                    z += torch.einsum("mk,nk->mn", s["x2"][b, r].double(), d["w"][:, c["K"]:])
                z += d.get("bias", 0.0 * one)
                if c["act"] == "silu":
                    z = z * torch.sigmoid(z)
                elif c["act"] == "swiglu":
                    z = z[:, :c["N"]] * torch.sigmoid(z[:, :c["N"]]) * z[:, c["N"]:]
                elif c["act"] == "gelu_tanh":
                    z = z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
                z = z * (d["gate"][b] if c["gate"] else one)
                parts.append((z + (s["residual"][b, r].double() if c["residual"] else 0.0 * one),))
            else:
                if c["y"]:
                    x = torch.addcmul(x, s["y"][b, r].double(), d["gate"][b])
                t = x if c["kind"] == "rms" else x - x.sum(-1, keepdim=True) / c["dim"]
                h = t * torch.rsqrt(t.pow(2).sum(-1, keepdim=True) / c["dim"] + EPS)
                if c["modulated"]:
                    h = torch.addcmul(d["shift"][b] + h, h, d["scale"][b])
                parts.append((h, x) if c["y"] else (h,))
    outs = tuple(torch.cat(p).reshape(c["B"], c["S"], -1) for p in zip(*parts))
    return outs[0] if len(outs) == 1 else outs
