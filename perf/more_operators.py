"""Cases for measuring a block's cross-attention and its products in 8-bit floating point.

Three operators, each in a plain form (elementary torch operations in fp32, one
rounding at the end) and, with ``own`` set, as a user calls them:

- ``quantize``: rows or a weight to e4m3 values with an fp32 scale per group of
  128 channels of a row (activations) or per 128 x 128 block (weights):
  scale = max |x| / 448, q = e4m3(x * (448 / max |x|)).
- ``linear``: out = residual + gate * act(x W^T + bias) with x and W in e4m3
  and those scales.
- ``cross``: softmax(scale q k^T) v of image tokens (or a few queries) over an
  encoder's states of another length, padded to their batch's longest:
  ``lengths`` or a ``mask`` say which keys there are; heads may share keys and
  values. A row that no key is left for is zero.

Shapes follow the workloads of this repository (hidden widths 4096 and 6144,
MLP width three times that, 32 and 48 heads of 128, 512 text tokens, 4096 image
tokens, 12800 tokens in the two-reference edit) and prompts of 77 tokens.
"""
import math

import torch

own = False

BF16, F32 = "bfloat16", "float32"
TOP = 448.0  # the largest e4m3 value
LEAST = 2.0 ** -100  # a group's scale is at least that of this maximum


def _quantize(name, B, S, K, rows=1, x=BF16, strided=False):
    return {"op": "quantize", "name": name, "B": B, "S": S, "K": K, "rows": rows, "x": x,
            "strided": strided}


def _linear(name, B, S, K, N, act="none", bias=False, gate=False, residual=False, vec=BF16,
            strided=False):
    return {"op": "linear", "name": name, "B": B, "S": S, "K": K, "N": N, "act": act,
            "bias": bias, "gate": gate, "residual": residual, "vec": vec, "strided": strided}


def _cross(name, B, Sq, Sk, H, Hk, D=128, keys="all", strided=False):
    return {"op": "cross", "name": name, "B": B, "Sq": Sq, "Sk": Sk, "H": H, "Hk": Hk, "D": D,
            "keys": keys, "strided": strided}


def listed():
    return [
        # the encoder's states of a guided pair, before the key and value product
        _quantize("encoder_states", 2, 77, 4096),
        # the image stream after its norm
        _quantize("image_rows", 1, 4096, 4096),
        # a feed-forward weight, once when a model is loaded
        _quantize("weight_blocks", 1, 12288, 4096, rows=128),
        # second layer of the timestep MLP: one token
        _linear("one_token", 1, 1, 4096, 4096, bias=True),
        # keys and values of a guided pair's prompts, side by side
        _linear("prompt_kv", 2, 77, 4096, 8192, bias=True, vec=F32),
        # the image stream's attention output, gated onto the residual
        _linear("image_attn_out", 1, 4096, 4096, 4096, gate=True, residual=True),
        # the image stream's gated feed-forward in (a 52 x 78 grid)
        _linear("image_ff_in", 1, 4056, 4096, 12288, act="swiglu"),
        # the widest model's feed-forward out, two references
        _linear("edit_ff_out", 1, 12800, 18432, 6144, gate=True, residual=True),
        # one pooled query over the edit's image tokens, four query heads to a key head
        _cross("pooled_query", 1, 1, 12800, 32, 8, keys="mask"),
        # 64 learned queries over the image tokens, keys and values side by side
        _cross("few_queries", 2, 64, 4096, 32, 32, strided=True),
        # image tokens over a guided pair's prompts, padded to 512
        _cross("image_over_prompt", 2, 4056, 512, 32, 32, keys="lengths", strided=True),
        # the edit's tokens over the states of a long document
        _cross("edit_over_document", 1, 12800, 4096, 48, 48),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MOST_FLOPS = 2.0 * 12800 * 18432 * 6144
MOST_SCORES = 48 * 12800 * 4096


def draw(rng):
    """Sizes over the ranges of the listed cases, no costlier than the largest of them."""
    while True:
        kind = rng.random()
        if kind < 0.25:
            rows = rng.choice((1, 1, 128))
            c = _quantize("", 1 if rows > 1 else rng.choice((1, 1, 2, 3)), _log(rng, 1, 12800),
                          16 * _log(rng, 8, 1152), rows=rows, x=rng.choice((BF16, BF16, F32)),
                          strided=rng.random() < 0.4)
        elif kind < 0.65:
            act = rng.choice(("none", "none", "silu", "gelu_tanh", "swiglu"))
            n = 128 * _log(rng, 1, 144) if act == "swiglu" else 8 * _log(rng, 8, 2304)
            c = _linear("", rng.choice((1, 1, 2, 3)), _log(rng, 1, 12800), 16 * _log(rng, 8, 1152),
                        n, act=act, bias=rng.random() < 0.5, gate=rng.random() < 0.5,
                        residual=rng.random() < 0.5, vec=rng.choice((BF16, F32)),
                        strided=rng.random() < 0.4)
        else:
            hk = rng.choice((2, 5, 8, 16, 32))
            c = _cross("", rng.choice((1, 1, 2, 4)), _log(rng, 1, 12800), _log(rng, 1, 12800),
                       hk * rng.choice((1, 1, 1, 2, 3)), hk, D=rng.choice((128, 128, 64)),
                       keys=rng.choice(("all", "lengths", "mask")), strided=rng.random() < 0.4)
            if c["B"] * c["H"] * c["Sq"] * c["Sk"] > MOST_SCORES:
                continue
        if work(c)["flops"] <= MOST_FLOPS:
            del c["name"]
            return c


def work(c):
    """Bytes read and written once, and the operations of the products."""
    if c["op"] == "quantize":
        n = c["B"] * c["S"] * c["K"]
        groups = c["B"] * -(-c["S"] // c["rows"]) * -(-c["K"] // 128)
        return {"bytes": n * ((2 if c["x"] == BF16 else 4) + 1) + 4 * groups, "flops": 3 * n}
    if c["op"] == "linear":
        rows, K, N = c["B"] * c["S"], c["K"], c["N"]
        wr = 2 * N if c["act"] == "swiglu" else N
        kb = -(-K // 128)
        b = rows * K + wr * K + 4 * kb * (rows + -(-wr // 128))
        b += 2 * rows * N * (2 if c["residual"] else 1)
        vb = 2 if c["vec"] == BF16 else 4
        b += vb * ((wr if c["bias"] else 0) + (c["B"] * N if c["gate"] else 0))
        return {"bytes": b, "flops": 2 * rows * wr * K}
    # the first batch element has every key, another one of a padded batch 9/16 of them on average
    q, keys = c["B"] * c["Sq"] * c["H"] * c["D"], c["B"] * c["Sk"]
    if c["keys"] != "all":
        keys = c["Sk"] * (1 + (c["B"] - 1) * 9 / 16)
    b = 2 * (2 * q + 2 * keys * c["Hk"] * c["D"])
    b += {"all": 0, "lengths": 4 * c["B"], "mask": c["B"] * c["Sk"]}[c["keys"]]
    return {"bytes": b, "flops": 4 * c["Sq"] * c["H"] * c["D"] * keys}


def _channels(g, width):
    """Channel magnitudes as a network's activations have them: a few are several times the rest."""
    return torch.exp(0.6 * torch.randn(width, generator=g, device="cuda"))


def _rows(c, g, S, width, dtype, scale=None):
    """[B, S, width] rows; the trailing rows of a longer joint buffer when strided."""
    pad = 24 if c["strided"] else 0
    t = torch.randn((c["B"], pad + S, width), generator=g, device="cuda")
    if scale is not None:
        t *= scale
    return t.to(dtype)[:, pad:]


def _groups(x, rows):
    """|x|'s maximum per group of `rows` rows and 128 channels, at least LEAST, and the same
    spread over the group: x is [B, S, K] in fp32 or fp64."""
    B, S, K = x.shape
    sb, kb = -(-S // rows), -(-K // 128)
    a = torch.nn.functional.pad(x.abs(), (0, kb * 128 - K, 0, sb * rows - S))
    top = a.reshape(B, sb, rows, kb, 128).amax(dim=(2, 4)).clamp(min=LEAST)
    wide = top.repeat_interleave(rows, 1)[:, :S].repeat_interleave(128, 2)[:, :, :K]
    return top, wide


def _to_e4m3(x, rows):
    """(e4m3 values, fp32 scales per group), in fp32."""
    top, wide = _groups(x.float(), rows)
    # (a number over a tensor would be its reciprocal's multiple, rounded twice)
    q = x.float() * (torch.full_like(wide, TOP) / wide)
    return q.to(torch.float8_e4m3fn), top / TOP


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    bf16 = torch.bfloat16
    s = {"case": dict(c)}
    if c["op"] == "quantize":
        xt = getattr(torch, c["x"])
        if c["rows"] == 1:
            s["x"] = _rows(c, g, c["S"], c["K"], xt, _channels(g, c["K"]))
        else:
            s["x"] = _rows(c, g, c["S"], c["K"], xt, c["K"] ** -0.5)[0]
        lead = tuple(s["x"].shape[:-1])
        s["q"] = torch.empty(lead + (c["K"],), dtype=torch.float8_e4m3fn, device="cuda")
        return s
    if c["op"] == "linear":
        B, S, K, N, vec = c["B"], c["S"], c["K"], c["N"], getattr(torch, c["vec"])
        wr = 2 * N if c["act"] == "swiglu" else N
        x = torch.randn((B, S, K), generator=g, device="cuda") * _channels(g, K)
        s["x"], xs = _to_e4m3(x.to(bf16), 1)
        # a group's scales of all tokens lie beside one another, as the quantisation leaves them
        flat = xs.reshape(B * S, -1).T.contiguous()
        s["xs"] = flat.reshape(-1, B, S).permute(1, 2, 0)
        w = torch.randn((1, wr, K), generator=g, device="cuda") * K ** -0.5
        w, ws = _to_e4m3(w, 128)
        s["w"], s["ws"] = w[0], ws[0]
        s["bias"] = (0.2 * torch.randn(wr, generator=g, device="cuda")).to(vec) if c["bias"] else None
        s["gate"] = (0.5 * torch.randn((B, N), generator=g, device="cuda")).to(vec) \
            if c["gate"] else None
        s["residual"] = _rows(c, g, S, N, bf16, _channels(g, N)) if c["residual"] else None
        s["out"] = _rows(c, g, S, N, bf16)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    B, Sq, Sk, H, Hk, D = (c[k] for k in ("B", "Sq", "Sk", "H", "Hk", "D"))
    s["q"] = _rows(c, g, Sq, H * D, bf16).unflatten(-1, (H, D))
    # keys and values side by side, as one product leaves them, or apart
    if c["strided"]:
        kv = torch.randn((B, Sk, 2, Hk, D), generator=g, device="cuda").to(bf16)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
    else:
        s["k"], s["v"] = (torch.randn((B, Sk, Hk, D), generator=g, device="cuda").to(bf16)
                          for _ in range(2))
    # the longest prompt of the batch sets Sk, the others are padded
    lengths = torch.randint(max(1, Sk // 8), Sk + 1, (B,), generator=g, device="cuda")
    lengths[0] = Sk
    s["lengths"] = lengths.to(torch.int32) if c["keys"] == "lengths" else None
    s["mask"] = None
    if c["keys"] == "mask":  # padding in front of the shorter ones, and tokens left out
        at = torch.arange(Sk, device="cuda")
        keep = torch.rand((B, Sk), generator=g, device="cuda") < 0.9
        keep[:, -1] = True
        s["mask"] = keep & (at >= Sk - lengths[:, None])
    s["out"] = torch.empty((B, Sq, H, D), dtype=bf16, device="cuda")
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _run_own(s):
    from diffusion_transformer_joint_gb300 import binding

    c = s["case"]
    if c["op"] == "quantize":
        return binding.quantize_fp8(s["x"], rows=c["rows"], out=s["q"])
    if c["op"] == "linear":
        return binding.linear_fp8(s["x"], s["xs"], s["w"], s["ws"], bias=s["bias"],
                                  act=None if c["act"] == "none" else c["act"], gate=s["gate"],
                                  residual=s["residual"], out=s["out"], status=s["status"])
    return binding.cross_attention(s["q"], s["k"], s["v"], lengths=s["lengths"], mask=s["mask"],
                                   out=s["out"], status=s["status"])


def _plain_quantize(s):
    c = s["case"]
    x = s["x"] if s["x"].dim() == 3 else s["x"][None]
    q, scale = _to_e4m3(x, c["rows"])
    return (q, scale) if s["x"].dim() == 3 else (q[0], scale[0])


def _values(q, scale, rows):
    """The values that e4m3 rows [B, S, K] and their scales stand for, in fp32."""
    wide = scale.repeat_interleave(rows, 1)[:, :q.shape[1]].repeat_interleave(128, 2)
    return q.float() * wide[:, :, :q.shape[2]]


def _plain_linear(s):
    c = s["case"]
    y = _values(s["x"], s["xs"], 1) @ _values(s["w"][None], s["ws"][None], 128)[0].T
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


def _taken(s):
    """[B, Sk]: the keys that take part."""
    B, Sk = s["k"].shape[:2]
    if s["lengths"] is not None:
        return torch.arange(Sk, device="cuda") < s["lengths"][:, None]
    return s["mask"] if s["mask"] is not None else torch.ones((B, Sk), dtype=bool, device="cuda")


def _plain_cross(s):
    c = s["case"]
    B, Sq, Sk, H, Hk, D = (c[k] for k in ("B", "Sq", "Sk", "H", "Hk", "D"))
    q = s["q"].float().reshape(B, Sq, Hk, H // Hk, D).permute(0, 2, 3, 1, 4)
    k, v = (t.float().permute(0, 2, 1, 3)[:, :, None] for t in (s["k"], s["v"]))
    keep = _taken(s)
    p = (q * D ** -0.5) @ k.transpose(-1, -2)
    p = p.masked_fill(~keep[:, None, None, None], -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True).clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    v = v.masked_fill(~keep[:, None, None, :, None], 0.0)
    o = (p @ v) / torch.where(total > 0, total, 1.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, Sq, H, D).to(torch.bfloat16)


def run(state):
    if own:
        return _run_own(state)
    return {"quantize": _plain_quantize, "linear": _plain_linear,
            "cross": _plain_cross}[state["case"]["op"]](state)


def _nearest_e4m3(v):
    """v in fp64 rounded to the nearest e4m3 value, ties to even: steps of 2^-3 of the power of
    two below |v|, of 2^-9 below 2^-6."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(v / step) * step).clamp(-TOP, TOP)


def _exact_quantize(c, s):
    x = (s["x"] if s["x"].dim() == 3 else s["x"][None]).double()
    B, S, K = x.shape
    r, sb, kb = c["rows"], -(-S // c["rows"]), -(-K // 128)
    scale = torch.empty((B, sb, kb), dtype=torch.float64, device="cuda")
    q = torch.empty_like(x)
    for j in range(kb):
        part = x[:, :, 128 * j:128 * j + 128]
        top = part.abs().amax(-1)
        if r > 1:
            ids = torch.arange(S, device="cuda") // r
            block = torch.zeros((B, sb), dtype=torch.float64, device="cuda")
            block = block.index_reduce(1, ids, top, "amax")
            top, scale[:, :, j] = block[:, ids], block.clamp(min=LEAST) / TOP
        else:
            scale[:, :, j] = top.clamp(min=LEAST) / TOP
        q[:, :, 128 * j:128 * j + 128] = _nearest_e4m3(part * (TOP / top.clamp(min=LEAST))[..., None])
    return (q, scale) if s["x"].dim() == 3 else (q[0], scale[0])


def _exact_linear(c, s):
    K, N = c["K"], c["N"]
    kg = torch.arange(K, device="cuda") // 128
    wg = torch.arange(s["w"].shape[0], device="cuda") // 128
    w = s["w"].double() * s["ws"].double()[wg][:, kg]
    d = {k: s[k].double() for k in ("bias", "gate", "residual") if s[k] is not None}
    parts = []
    for b in range(c["B"]):
        for lo in range(0, c["S"], 1024):
            r = slice(lo, min(lo + 1024, c["S"]))
            z = torch.einsum("mk,nk->mn", s["x"][b, r].double() * s["xs"][b, r].double()[:, kg], w)
            if "bias" in d:
                z += d["bias"]
            if c["act"] == "silu":
                z = z * torch.sigmoid(z)
            elif c["act"] == "swiglu":
                z = z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:]
            elif c["act"] == "gelu_tanh":
                z = z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
            if "gate" in d:
                z = z * d["gate"][b]
            parts.append(z + d["residual"][b, r] if "residual" in d else z)
    return torch.cat(parts).reshape(c["B"], c["S"], N)


def _exact_cross(c, s):
    B, Sq, H, Hk, D = (c[k] for k in ("B", "Sq", "H", "Hk", "D"))
    out = torch.zeros((B, Sq, H, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        at = torch.arange(c["Sk"], device="cuda")
        if s["lengths"] is not None:
            at = at[:int(s["lengths"][b])]
        if s["mask"] is not None:
            at = at[s["mask"][b]]
        if at.numel() == 0:
            continue
        for h in range(H):
            k, v = (s[n][b, at, h * Hk // H].double() for n in ("k", "v"))
            w = torch.softmax(torch.einsum("id,jd->ij", s["q"][b, :, h].double(), k)
                              / math.sqrt(D), dim=-1)
            out[b, :, h] = torch.einsum("ij,jd->id", w, v)
    return out


def exact(case, seed):
    """The definitions in 64 bits, a group of channels, a range of rows or a head at a time."""
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "linear": _exact_linear,
            "cross": _exact_cross}[case["op"]](case, s)
