"""The measured cases of the 4-bit operators and of the mixture-of-experts layer for a few tokens.

Each case is one call path: a round trip through the 4-bit format (``quant``),
a product of two 4-bit operands (``gemm``; rows of one or several problems
stacked) and a whole mixture-of-experts layer (``moe``; 16-bit or 4-bit
weights).  With ``own`` false ``run`` computes it from elementary torch
operations in 32 bits; with ``own`` true it calls the framework.

4-bit format: blocks of 32 consecutive values of a row share one scale
2^(byte - 127), byte = max(0, exponent field of the block's largest magnitude
in 32 bits - 2); a value is held as the nearest (ties to even) of
{0, .5, 1, 1.5, 2, 3, 4, 6} times the scale, at most 6, with its sign.  A block
holding a NaN or an infinity has scale byte 255: all its values are NaN.
``codes`` [rows, 16 * blocks]: value 2i of a row in the low half of byte i,
value 2i + 1 in the high half.  ``scales`` [ceil(blocks / 8), rows, 8]: the
scales of 8 consecutive blocks of a row are neighbours.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
MAX_TOKENS = 64


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode batch's activations on their way into a 4-bit product: latency
        {"name": "quant 16x4096", "op": "quant", "rows": 16, "cols": 4096, "pad": 0, "dtype": "bf16"},
        # a ragged slice of a wider tensor: odd rows, a partial last block, rows not 16-byte aligned
        {"name": "quant ragged", "op": "quant", "rows": 1021, "cols": 2749, "pad": 14, "dtype": "fp16"},
        # one expert's weights, quantised once when a model is loaded
        {"name": "quant weights", "op": "quant", "rows": 28672, "cols": 8192, "pad": 0, "dtype": "bf16"},
        # one token through a tensor-parallel linear layer
        {"name": "gemm 1 token", "op": "gemm", "m": 1, "n": 8192, "k": 3584, "problems": 1, "dtype": "bf16"},
        # a decode batch through the same layer
        {"name": "gemm 128 tokens", "op": "gemm", "m": 128, "n": 8192, "k": 3584, "problems": 1, "dtype": "bf16"},
        # a short prompt: sizes that fit no tile
        {"name": "gemm ragged", "op": "gemm", "m": 777, "n": 4104, "k": 2752, "problems": 1, "dtype": "fp16"},
        # a prompt through a square layer
        {"name": "gemm prompt", "op": "gemm", "m": 2048, "n": 8192, "k": 8192, "problems": 1, "dtype": "bf16"},
        # a prompt's rows, sorted by expert, through the experts' first product
        {"name": "gemm experts", "op": "gemm", "m": 8192, "n": 14336, "k": 4096, "problems": 8, "dtype": "bf16"},
        # one token through a layer of 8 large experts, 16-bit weights
        {"name": "moe 1 token", "op": "moe", "tokens": 1, "hidden": 4096, "ffn": 14336, "experts": 8, "topk": 2,
         "first": 0, "local": 8, "weights": "16", "renorm": True, "dtype": "bf16"},
        # a decode batch through the same layer in 4 bits
        {"name": "moe 16 tokens mx4", "op": "moe", "tokens": 16, "hidden": 4096, "ffn": 14336, "experts": 8, "topk": 2,
         "first": 0, "local": 8, "weights": "mx4", "renorm": True, "dtype": "bf16"},
        # a few tokens through many small experts
        {"name": "moe small experts", "op": "moe", "tokens": 13, "hidden": 2048, "ffn": 776, "experts": 128, "topk": 8,
         "first": 0, "local": 128, "weights": "16", "renorm": True, "dtype": "fp16"},
        # one rank's share of the experts (expert parallel): many picks are elsewhere, some tokens have none here
        {"name": "moe share mx4", "op": "moe", "tokens": 64, "hidden": 2048, "ffn": 1408, "experts": 64, "topk": 6,
         "first": 16, "local": 8, "weights": "mx4", "renorm": False, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "moe", "moe"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "quant":
        cols = _log(rng, 33, 16384)
        rows = max(1, min(_log(rng, 1, 32768), 28672 * 8192 // cols))
        return {"op": op, "rows": rows, "cols": cols, "pad": rng.choice([0, 0, 8, rng.randrange(1, 40)]), "dtype": dtype}
    if op == "gemm":
        problems = rng.choice([1, 1, rng.randrange(2, 33)])
        while True:
            m, n, k = _log(rng, 1, 8192), 8 * _log(rng, 16, 1792), 32 * _log(rng, 4, 256)
            if problems * n * k <= 8 * 14336 * 4096:
                return {"op": op, "m": m, "n": n, "k": k, "problems": problems, "dtype": dtype}
    weights = rng.choice(["16", "mx4"])
    while True:
        step = 32 if weights == "mx4" else 8
        hidden, ffn = step * (_log(rng, 256, 4096) // step), step * (_log(rng, 128, 14336) // step)
        experts = _log(rng, 2, 256)
        local = experts if rng.random() < 0.7 else rng.randrange(1, experts + 1)
        tokens, topk = _log(rng, 1, MAX_TOKENS), rng.randrange(1, min(8, experts) + 1)
        if local * hidden * ffn <= 8 * 4096 * 14336 and (local == experts or tokens * topk * local >= 8 * experts):
            return {"op": op, "tokens": tokens, "hidden": hidden, "ffn": ffn, "experts": experts, "topk": topk,
                    "first": rng.randrange(0, experts - local + 1), "local": local, "weights": weights,
                    "renorm": rng.random() < 0.5, "dtype": dtype}


def _blocks(cols):
    return -(-cols // 32)


def work(case):
    if case["op"] == "quant":  # in, 4-bit form written and read again, out
        n = case["rows"] * case["cols"]
        return {"bytes": 4 * n + 2 * case["rows"] * _blocks(case["cols"]) * 17, "flops": 2 * n}
    if case["op"] == "gemm":
        m, n, k, p = case["m"], case["n"], case["k"], case["problems"]
        return {"bytes": (m + min(p, m) * n) * (k // 32) * 17 + 2 * m * n, "flops": 2 * m * n * k}
    t, d, f, e, j = case["tokens"], case["hidden"], case["ffn"], case["experts"], case["topk"]
    active = case["local"] * (1 - (1 - j / e) ** t)  # experts that at least one token picks, in the mean
    per = 2 if case["weights"] == "16" else 17 / 32
    return {"bytes": active * 3 * d * f * per + 2 * e * d + 4 * t * d, "flops": 2 * t * d * (e + 3 * f * j * case["local"] / e)}


# ------------------------------------------------------------------ the 4-bit format in elementary operations
def _codes_of(x):
    """fp32 [rows, 32 * blocks] -> (magnitudes 0 .. 6 [rows, blocks, 32], scale bytes [rows, blocks])."""
    b = x.view(x.shape[0], -1, 32)
    field = (b.abs().amax(-1).nan_to_num(nan=math.inf).view(torch.int32) >> 23) & 255
    byte = (field - 2).clamp_min(0)
    byte = torch.where(field == 255, 255, byte)
    y = b.abs() * ((254 - byte.clamp_max(253)) << 23).view(torch.float32)[..., None]
    y = torch.where(y < 2, torch.round(2 * y) / 2, torch.where(y < 4, torch.round(y), 2 * torch.round(y / 2))).clamp_max(6)
    return torch.where(byte[..., None] == 255, 0, y), byte


def _scale_of(byte):
    s = torch.where(byte == 0, 2.0 ** -127, (byte.to(torch.int32) << 23).view(torch.float32))
    return torch.where(byte == 255, math.nan, s)


def _round_trip(x, dtype):
    rows, cols = x.shape
    f = torch.nn.functional.pad(x.float(), (0, -cols % 32))
    y, byte = _codes_of(f)
    v = torch.copysign(y, f.view(rows, -1, 32)) * _scale_of(byte)[..., None]
    return v.view(rows, -1)[:, :cols].to(dtype)


def _pack(x):
    """fp32 [rows, cols], cols a multiple of 32 -> (codes, scales) as the framework lays them out."""
    y, byte = _codes_of(x)
    c = torch.where(y <= 2, 2 * y, torch.where(y <= 4, y + 2, 7)).to(torch.uint8)
    c = (c | (torch.signbit(x.view_as(y)).to(torch.uint8) << 3)).view(x.shape[0], -1, 2)
    byte = torch.nn.functional.pad(byte.to(torch.uint8), (0, -byte.shape[1] % 8))
    return c[..., 0] | (c[..., 1] << 4), byte.view(x.shape[0], -1, 8).transpose(0, 1).contiguous()


_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _unpack(codes, scales):
    """codes [..., rows, 16 * blocks] and scales [panels, ..., rows, 8] -> fp32 [..., rows, 32 * blocks]."""
    table = torch.tensor(_VALUES, device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).view(*codes.shape[:-1], -1, 32)
    s = _scale_of(scales).movedim(0, -2).flatten(-2)[..., : v.shape[-2]]
    return (v * s[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, cols):
    """Normal values with a few channels much larger than the rest, as a model's hidden states have."""
    x = _normal(g, rows, cols)
    x[:, torch.randint(0, cols, (1 + cols // 256,), generator=g, device="cuda")] *= 12
    return x


def _weights(g, rows, cols, kind, dtype):
    """Normal weights in 16 bits, or (codes, scales); a band of rows at a time, so that the 32-bit form stays small."""
    band = max(1, (1 << 27) // cols)
    made = []
    for r in range(0, rows, band):
        w = _normal(g, min(band, rows - r), cols) * cols ** -0.5
        made.append(w.to(dtype) if kind == "16" else _pack(w))
    if kind == "16":
        return torch.cat(made, 0)
    return torch.cat([m[0] for m in made], 0), torch.cat([m[1] for m in made], 1)


def _split(seed, m, problems):
    """Rows of each problem: uneven, the second of several left empty."""
    c = torch.rand(problems, generator=torch.Generator().manual_seed(seed)) + 0.2
    c[1] = 0 if problems > 2 else c[1]
    ends = torch.round(c.cumsum(0) / c.sum() * m).long().tolist()
    return ends[:-1] + [m]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "quant":
        rows, cols = case["rows"], case["cols"]
        wide = _activations(g, rows, cols + case["pad"])
        wide[torch.rand(rows, generator=g, device="cuda") < 0.02] = 0  # padding rows
        s["x"] = wide.to(dtype)[:, :cols]
        return s
    if case["op"] == "gemm":
        m, n, k, p = case["m"], case["n"], case["k"], case["problems"]
        s["a"] = _pack(_activations(g, m, k))
        s["b"] = _weights(g, p * n, k, "mx4", None)
        if p > 1:
            ends = _split(seed, m, p)
            counts = [e - b for b, e in zip([0] + ends[:-1], ends)]
            s["ends"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
            s["most"] = max(counts)
            s["place"] = torch.cat([torch.arange(c) + i * s["most"] for i, c in enumerate(counts)]).cuda()
        return s
    d, f, e, local = case["hidden"], case["ffn"], case["experts"], case["local"]
    s["x"] = _activations(g, case["tokens"], d).to(dtype)
    s["router"] = _weights(g, e, d, "16", dtype)
    s["gate_up"] = _weights(g, local * 2 * f, d, case["weights"], dtype)
    s["down"] = _weights(g, local * d, f, case["weights"], dtype)
    if own:  # the layer's description and its workspace, made once and kept beside the weights
        import gemm_tile_signaling_amd as fo
        s["layer"] = fo.Moe(d, f, e, case["topk"], dtype=case["dtype"], weights=case["weights"], renormalize=case["renorm"],
                            first_expert=case["first"], local_experts=local, max_tokens=MAX_TOKENS)
        s["workspace"] = s["layer"].new_workspace("cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import gemm_tile_signaling_amd as fo
    c = s["case"]
    if c["op"] == "quant":
        codes, scales = fo.mx4_quantize(s["x"])
        return fo.mx4_dequantize(codes, scales, c["cols"], dtype=c["dtype"])
    if c["op"] == "gemm":
        return fo.mx4_gemm(*s["a"], *s["b"], dtype=c["dtype"], row_ends=s.get("ends"))
    return s["layer"].forward(s["x"], s["router"], s["gate_up"], s["down"], s["workspace"])


def _plain(s):
    c = s["case"]
    dtype = _TYPES[c["dtype"]]
    if c["op"] == "quant":
        return _round_trip(s["x"], dtype)
    if c["op"] == "gemm":
        a, b = _unpack(*s["a"]), _unpack(*s["b"])
        if c["problems"] == 1:
            return (a @ b.t()).to(dtype)
        padded = torch.zeros(c["problems"] * s["most"], c["k"], device=a.device)
        padded[s["place"]] = a
        out = torch.matmul(padded.view(c["problems"], -1, c["k"]), b.view(c["problems"], -1, c["k"]).transpose(1, 2))
        return out.view(-1, c["n"])[s["place"]].to(dtype)
    t, d, f, k, local = c["tokens"], c["hidden"], c["ffn"], c["topk"], c["local"]
    x = s["x"].float()
    logits = x @ s["router"].float().t()
    ids = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(logits, -1).gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    here = (ids >= c["first"]) & (ids < c["first"] + local)
    at, w = (ids - c["first"]).clamp(0, local - 1), torch.where(here, w, 0)
    few = t * k < local  # fewer picks than experts: the picks' weights alone are taken
    wide = lambda m, rows: (_picked(m, rows, local, at.flatten()) if few else _stacked(m, rows, local))  # noqa: E731
    if few:
        h = torch.matmul(wide(s["gate_up"], 2 * f), x.repeat_interleave(k, 0)[..., None])[..., 0]
        y = torch.matmul(wide(s["down"], d), (_silu(h[:, :f]) * h[:, f:])[..., None])[..., 0].view(t, k, d)
        return (w[..., None] * y).sum(1).to(dtype)
    h = torch.matmul(x, wide(s["gate_up"], 2 * f).transpose(1, 2))
    y = torch.matmul(_silu(h[..., :f]) * h[..., f:], wide(s["down"], d).transpose(1, 2))
    share = torch.zeros(t, local, device=x.device).scatter_add_(1, at, w)
    return (share.t()[..., None] * y).sum(0).to(dtype)


def _silu(v):
    return v / (1 + torch.exp(-v))


def _stacked(m, rows, local):
    if isinstance(m, torch.Tensor):
        return m.view(local, rows, -1).float()
    return _unpack(m[0].view(local, rows, -1), m[1].view(-1, local, rows, 8))


def _picked(m, rows, local, at):
    if isinstance(m, torch.Tensor):
        return m.view(local, rows, -1)[at].float()
    return _unpack(m[0].view(local, rows, -1)[at], m[1].view(-1, local, rows, 8)[:, at])


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "quant":
        x = s["x"].double()
        out = torch.empty_like(x)
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
        middle = (grid[1:] + grid[:-1]) / 2
        even = torch.tensor([True, False, True, False, True, False, True], device=x.device)  # a tie goes to the even code
        for c in range(0, x.shape[1], 32):
            b = x[:, c:c + 32]
            top = b.abs().amax(1, keepdim=True)
            e = (torch.frexp(top).exponent - 3).clamp_min(-127)  # floor(log2 top) - 2
            scale = torch.where(top > 0, torch.pow(2.0, e.double()), 2.0 ** -127)
            y = (b.abs() / scale)[..., None]
            code = torch.where(even, y > middle, y >= middle).sum(-1)
            out[:, c:c + 32] = torch.sign(b) * grid[code] * scale
        return out
    if case["op"] == "gemm":
        a, n, p = _exact_values(*s["a"]), case["n"], case["problems"]
        ends = s["ends"].tolist() if p > 1 else [case["m"]]
        out, begin = [], 0
        for i, end in enumerate(ends):
            if end > begin:
                out.append(a[begin:end] @ _exact_values(s["b"][0][i * n:(i + 1) * n], s["b"][1][:, i * n:(i + 1) * n]).t())
            begin = end
        return torch.cat(out)
    x, f, d = s["x"].double(), case["ffn"], case["hidden"]
    logits = x @ s["router"].double().t()
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    ids = torch.argsort(logits, dim=-1, descending=True, stable=True)[:, : case["topk"]]
    chosen = torch.zeros_like(p).scatter_(1, ids, 1.0) * p
    if case["renorm"]:
        chosen = chosen / chosen.sum(-1, keepdim=True)
    part = lambda m, i, rows: (m[i * rows:(i + 1) * rows].double() if isinstance(m, torch.Tensor)  # noqa: E731
                               else _exact_values(m[0][i * rows:(i + 1) * rows], m[1][:, i * rows:(i + 1) * rows]))
    out = torch.zeros_like(x)
    for i in range(case["local"]):
        g, u = (x @ part(s["gate_up"], i, 2 * f).t()).split(f, -1)
        out += chosen[:, case["first"] + i, None] * ((g * torch.sigmoid(g) * u) @ part(s["down"], i, d).t())
    return out


def _exact_values(codes, scales):
    rows = codes.shape[0]
    nibble = torch.stack((codes % 16, codes // 16), -1).reshape(rows, -1).long()
    e, m = (nibble % 8) // 2, (nibble % 2).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, (e - 1).double()))
    v = torch.where(nibble >= 8, -v, v)
    byte = scales.transpose(0, 1).reshape(rows, -1)[:, : v.shape[1] // 32].double()
    return v * torch.pow(2.0, byte - 127).repeat_interleave(32, 1)
