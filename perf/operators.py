"""The MXFP4 operators and the MoE router: what is measured, and their plain forms.

Five operators of a mixture-of-experts engine whose routed experts are held in
MXFP4 (blocks of 32 e2m1 values under one e8m0 scale): quantisation of
activations, dequantisation, the product of two MXFP4 matrices, the top-k
router, and the whole layer for a few tokens.  `run` computes them in
elementary torch operations in 32 bits, or, where `own` is true, through the
framework's calls.

Quantised values are compared as the values that they stand for, so the
quantiser is measured together with the dequantiser (a round trip, exact in
bfloat16).
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---- cases ---------------------------------------------------------------

def listed():
    return [
        # One decode token's hidden state: the launch itself is the cost.
        {"name": "quant_decode_1x4096", "op": "quant", "rows": 1, "k": 4096, "pad": 0, "dtype": "fp32"},
        # A ragged batch of rows cut out of a wider fused projection (row stride above the row).
        {"name": "quant_rows_777x1056", "op": "quant", "rows": 777, "k": 1056, "pad": 96, "dtype": "fp16"},
        # The widest activation rows of the engine at prefill (attention output, 2048 tokens).
        {"name": "quant_prefill_2048x32768", "op": "quant", "rows": 2048, "k": 32768, "pad": 0, "dtype": "bf16"},
        # The decode projection of a single token with the most rows.
        {"name": "mm_decode_1024x32768_1", "op": "mm", "k": 1024, "n": 32768, "t": 1, "out": "fp32"},
        # A few sequences decoding together, sizes that fill no tile: ragged rows, K not a multiple of 128.
        {"name": "mm_odd_2912x1000_13", "op": "mm", "k": 2912, "n": 1000, "t": 13, "out": "bf16"},
        # A mid-size batch: between the weight-bound and the matrix-core-bound ends.
        {"name": "mm_batch_4096x2048_200", "op": "mm", "k": 4096, "n": 2048, "t": 200, "out": "bf16"},
        # Prefill with a long K and few output rows.
        {"name": "mm_prefill_32768x1024_2048", "op": "mm", "k": 32768, "n": 1024, "t": 2048, "out": "fp32"},
        # The router of 64 tokens decoding together (256 experts, 8 a token).
        {"name": "topk_64x256_8", "op": "topk", "t": 64, "e": 256, "u": 8, "scoring": "softmax", "bias": False, "renorm": True},
        # The router at prefill, with a load-balancing bias on the selection.
        {"name": "topk_4096x256_8_bias", "op": "topk", "t": 4096, "e": 256, "u": 8, "scoring": "sqrt_softplus", "bias": True, "renorm": True},
        # The layer for one token: the latency of a decode step.
        {"name": "layer_1_4096x2048_e256", "op": "layer", "t": 1, "d": 4096, "f": 2048, "e": 256, "u": 8, "scoring": "softmax", "bias": False, "renorm": True,
         "clamp": 0.0, "masked": 0, "x": "bf16", "out": "bf16"},
        # A handful of tokens, odd widths, few experts shared by several tokens, some rows of the batch empty.
        {"name": "layer_11_1056x352_e20", "op": "layer", "t": 11, "d": 1056, "f": 352, "e": 20, "u": 4, "scoring": "sigmoid", "bias": True, "renorm": True,
         "clamp": 10.0, "masked": 2, "x": "fp32", "out": "fp16"},
        # 64 tokens decoding together: nearly every expert is touched.
        {"name": "layer_64_4096x2048_e256", "op": "layer", "t": 64, "d": 4096, "f": 2048, "e": 256, "u": 8, "scoring": "softmax", "bias": False, "renorm": True,
         "clamp": 10.0, "masked": 0, "x": "bf16", "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "mm", "topk", "layer"))
    if op == "quant":
        k = BLOCK * _log_int(rng, 1, 1024)
        rows = _log_int(rng, 1, max(1, min(65536, (2048 * 32768) // k)))
        return {"op": op, "rows": rows, "k": k, "pad": rng.choice((0, 0, 8, 96)), "dtype": rng.choice(("fp32", "bf16", "fp16"))}
    if op == "mm":
        k = BLOCK * _log_int(rng, 2, 1024)
        n = _log_int(rng, 16, 32768)
        room = 32768 * 1024 * 2048 // (k * n)
        t = _log_int(rng, 1, max(1, min(4096, room)))
        return {"op": op, "k": k, "n": n, "t": t, "out": rng.choice(("fp32", "bf16", "fp16"))}
    e = _log_int(rng, 8, 512 if op == "topk" else 256)
    u = rng.randint(1, 8)
    route = {"e": e, "u": u, "scoring": rng.choice(("softmax", "sigmoid", "sqrt_softplus")), "bias": rng.random() < 0.5, "renorm": rng.random() < 0.7}
    if op == "topk":
        return {"op": op, "t": _log_int(rng, 1, 2048), **route}
    d, f, t = BLOCK * _log_int(rng, 8, 128), BLOCK * _log_int(rng, 4, 64), _log_int(rng, 1, 64)
    return {"op": op, "t": t, "d": d, "f": f, **route, "clamp": rng.choice((0.0, 10.0)), "masked": rng.choice((0, t // 5)), "x": rng.choice(("fp32", "bf16", "fp16")),
            "out": rng.choice(("bf16", "fp16"))}


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["k"]
        # the input once, the codes and scales once, the values that they stand for once
        return {"bytes": n * (4 if case["dtype"] == "fp32" else 2) + n * 17 // 32 + n * 2, "flops": 4 * n}
    if op == "mm":
        k, n, t = case["k"], case["n"], case["t"]
        return {"bytes": (n + t) * k * 17 // 32 + n * t * (4 if case["out"] == "fp32" else 2), "flops": 2 * n * t * k}
    t, e, u = case["t"], case["e"], min(case["u"], case["e"])
    route = t * e * 4 + t * u * 8
    if op == "topk":
        return {"bytes": route, "flops": 8 * t * e}
    d, f = case["d"], case["f"]
    real = t - case["masked"]
    touched = e * (1.0 - (1.0 - u / e) ** real)  # distinct experts, expected
    return {"bytes": int(touched * 3 * d * f * 17 / 32) + t * d * ((4 if case["x"] == "fp32" else 2) + 2) + route, "flops": real * u * 6 * d * f}


# ---- inputs --------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _weights(shape, g):
    """(codes, scales) of normal weights, a slice of the first axis at a time."""
    rows, k = math.prod(shape[:-1]), shape[-1]
    codes = torch.empty((rows, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, k // BLOCK), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // k)
    for i in range(0, rows, step):
        c, s = _encode(torch.randn((min(step, rows - i), k), generator=g, device="cuda").mul_(0.02))
        codes[i:i + step], scales[i:i + step] = c, s
    return codes.view(*shape[:-1], k // 2), scales.view(*shape[:-1], k // BLOCK)


def _activations(rows, k, g):
    """N(0, 1) with 1% of the channels 20 times larger, as activations have."""
    x = torch.randn((rows, k), generator=g, device="cuda")
    loud = torch.rand((k,), generator=g, device="cuda") < 0.01
    return x * (1.0 + 19.0 * loud)


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    op = case["op"]
    if op == "quant":
        x = _activations(case["rows"], case["k"] + case["pad"], g).to(DTYPES[case["dtype"]])
        s["x"] = x[:, :case["k"]]
    elif op == "mm":
        s["w"] = _weights((case["n"], case["k"]), g)
        s["x"] = _encode(_activations(case["t"], case["k"], g))
    else:
        t, e = case["t"], case["e"]
        s["logits"] = torch.randn((t, e), generator=g, device="cuda") * 1.5
        s["bias"] = torch.randn((e,), generator=g, device="cuda") * 0.1 if case["bias"] else None
        if op == "layer":
            d, f = case["d"], case["f"]
            s["logits"][t - case["masked"]:] = -math.inf  # the padded end of the batch
            s["x"] = _activations(t, d, g).to(DTYPES[case["x"]])
            s["gate"], s["up"], s["down"] = _weights((e, f, d), g), _weights((e, f, d), g), _weights((e, d, f), g)
    if own:
        import q8_quantized_matmul_amd as q8
        if op == "mm":  # a program keeps the scratch of its shapes
            s["w"], s["x"] = q8.Mxfp4(*s["w"]), q8.Mxfp4(*s["x"])
            s["workspace"] = q8.mxfp4_matmul_workspace(case["k"], case["n"], case["t"])
        if op == "layer":
            s["gate"], s["up"], s["down"] = (q8.Mxfp4(*s[m]) for m in ("gate", "up", "down"))
            s["workspace"] = q8.mxfp4_moe_layer_workspace(case["t"], min(case["u"], case["e"]), case["e"], case["d"], case["f"])
    return s


# ---- the plain forms -----------------------------------------------------

def _power(e):
    """2^e in fp32 for whole e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _encode(x):
    """Codes (two a byte, the even value in the low half) and scale bytes of fp32 rows.  Shared exponent floor(log2(amax)) - 2, values rounded to
    nearest with ties to even and held at +-6."""
    rows, k = x.shape
    b = x.view(rows, k // BLOCK, BLOCK)
    amax = b.abs().amax(-1)
    shared = torch.where(amax > 0, torch.frexp(amax).exponent.to(torch.int32) - 3, -127).clamp(min=-127)
    a = b * _power(-shared).unsqueeze(-1)
    m = a.abs()
    c = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)) + 8 * torch.signbit(a).to(torch.uint8)
    c = c.view(rows, k // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), (shared + 127).to(torch.uint8)


def _decode(codes, scales):
    """The fp32 values that codes [..., k/2] and scales [..., k/32] stand for."""
    pairs = torch.tensor([[E2M1[i & 15], E2M1[i >> 4]] for i in range(256)], device=codes.device)
    v = pairs[codes.to(torch.int32)].view(*scales.shape, BLOCK)
    half = _power(scales.to(torch.int32) - 127 + 1)  # 2^-126 .. : twice the scale, so that the smallest stays normal
    return (v * 0.5 * half.unsqueeze(-1)).view(*codes.shape[:-1], codes.shape[-1] * 2)


def _select(logits, bias, u, scoring, renorm):
    """(ids, weights): the u experts of the largest score + bias, and their scores."""
    z = logits
    if scoring == "softmax":
        key = z if bias is None else z + bias
    else:  # in 64 bits: the border between two experts decides which is taken
        z = z.double()
        key = torch.sigmoid(z) if scoring == "sigmoid" else torch.log1p(torch.exp(-z.abs())).add(z.clamp(min=0)).sqrt()
        key = key if bias is None else key + bias
    order = torch.sort(torch.where(logits > -math.inf, key, -math.inf), dim=-1, descending=True, stable=True)
    ids = order.indices[:, :u]
    taken = order.values[:, :u] > -math.inf
    if scoring == "softmax":
        top = logits.amax(-1, keepdim=True)
        p = torch.exp(logits - torch.where(top > -math.inf, top, 0.0))
        w = torch.where(taken, torch.gather(p, 1, ids), 0.0)
        total = (w if renorm else p).sum(-1, keepdim=True)
    else:
        p = torch.sigmoid(z) if scoring == "sigmoid" else torch.log1p(torch.exp(-z.abs())).add(z.clamp(min=0)).sqrt()
        w = torch.where(taken, torch.gather(p, 1, ids), 0.0).float()
        total = w.sum(-1, keepdim=True) if renorm else torch.ones_like(w[:, :1])
    return torch.where(taken, ids, -1).to(torch.int32), w / torch.where(total > 0, total, 1.0)


def _pair_product(m, ids, rows):
    """Each (token, slot)'s expert matrix times its row: [p, n, k] x [p, k]."""
    w = _decode(m[0][ids], m[1][ids])
    return torch.bmm(w, rows.unsqueeze(-1)).squeeze(-1)


def _layer(s):
    c = s["case"]
    t, u = c["t"], min(c["u"], c["e"])
    ids, weights = _select(s["logits"], s["bias"], u, c["scoring"], c["renorm"])
    flat = ids.reshape(-1).clamp(min=0).long()
    x = _decode(*_encode(s["x"].float())).repeat_interleave(u, 0)
    gate, up = _pair_product(s["gate"], flat, x), _pair_product(s["up"], flat, x)
    if c["clamp"] > 0:
        gate, up = gate.clamp(max=c["clamp"]), up.clamp(-c["clamp"], c["clamp"])
    mid = gate / (1.0 + torch.exp(-gate)) * up
    y = _pair_product(s["down"], flat, _decode(*_encode(mid))).view(t, u, c["d"])
    out = (torch.where(ids >= 0, weights, 0.0).unsqueeze(-1) * y).sum(1)
    return out.to(DTYPES[c["out"]]), ids, weights


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import q8_quantized_matmul_amd as q8
        if op == "quant":
            return q8.mxfp4_dequantize(q8.mxfp4_quantize(s["x"]), dtype=torch.bfloat16)
        if op == "mm":
            return q8.mxfp4_matmul(s["w"], s["x"], out_dtype=DTYPES[c["out"]], workspace=s["workspace"])
        scoring = {"softmax": q8.MOE_SOFTMAX, "sigmoid": q8.MOE_SIGMOID, "sqrt_softplus": q8.MOE_SQRT_SOFTPLUS}[c["scoring"]]
        u = min(c["u"], c["e"])
        if op == "topk":
            return q8.moe_topk(s["logits"], u, bias=s["bias"], scoring=scoring, renormalize=c["renorm"])
        return q8.mxfp4_moe_layer(s["x"], s["logits"], s["gate"], s["up"], s["down"], u, bias=s["bias"], scoring=scoring, renormalize=c["renorm"],
                                  clamp=c["clamp"], out_dtype=DTYPES[c["out"]], workspace=s["workspace"])
    if op == "quant":
        return _decode(*_encode(s["x"].float())).to(torch.bfloat16)
    if op == "mm":
        return torch.mm(_decode(*s["x"]), _decode(*s["w"]).t()).to(DTYPES[c["out"]])
    if op == "topk":
        return _select(s["logits"], s["bias"], min(c["u"], c["e"]), c["scoring"], c["renorm"])
    return _layer(s)


# ---- the definition in 64 bits -------------------------------------------

def _values64(codes, scales):
    """sign * (mantissa of the code) * 2^(scale - 127), from the bits."""
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).to(torch.int16)
    e, m = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2((e - 1).double()))
    scale = torch.exp2(scales.double() - 127.0).repeat_interleave(BLOCK, -1)
    return torch.where(nib >= 8, -mag, mag) * scale


def _quantised64(x):
    """x rounded to the block format: the nearest multiple of each binade's step, in doubles."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.clamp(torch.frexp(torch.where(amax > 0, amax, 1.0)).exponent.double() - 3.0, min=-127.0))
    a = (b / scale).clamp(-6.0, 6.0)
    step = torch.where(a.abs() < 2.0, 0.5, torch.where(a.abs() < 4.0, 1.0, 2.0))
    return (torch.round(a / step) * step * scale * (amax > 0)).flatten(-2)


def _routing64(s, u):
    c = s["case"]
    z = s["logits"].double()
    live = z > -math.inf
    if c["scoring"] == "softmax":
        score = torch.softmax(torch.where(live, z, -1e300), -1) * live
        key = z
    else:
        score = (1.0 / (1.0 + torch.exp(-z)) if c["scoring"] == "sigmoid" else torch.sqrt(torch.logaddexp(z, torch.zeros_like(z)))) * live
        key = score
    if s["bias"] is not None:
        key = (s["logits"] + s["bias"]).double() if c["scoring"] == "softmax" else key + s["bias"].double()
    key = torch.where(live, key, -math.inf)
    ids = torch.argsort(key, dim=-1, descending=True, stable=True)[:, :u]
    taken = torch.gather(live, 1, ids)
    w = torch.gather(score, 1, ids) * taken
    if c["renorm"]:
        w = w / torch.where(w.sum(-1, keepdim=True) > 0, w.sum(-1, keepdim=True), 1.0)
    return torch.where(taken, ids, -1), w


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return _quantised64(s["x"])
    if op == "mm":
        w, x = _values64(*s["w"]), _values64(*s["x"])
        return torch.matmul(x, w.transpose(0, 1).contiguous())
    u = min(case["u"], case["e"])
    ids, w = _routing64(s, u)
    if op == "topk":
        return ids.to(torch.int32), w
    x = _quantised64(s["x"])
    out = torch.zeros((case["t"], case["d"]), dtype=torch.float64, device="cuda")
    for e in torch.unique(ids[ids >= 0]).tolist():  # an expert at a time
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        g = x[tok] @ _values64(s["gate"][0][e], s["gate"][1][e]).t().contiguous()
        v = x[tok] @ _values64(s["up"][0][e], s["up"][1][e]).t().contiguous()
        if case["clamp"] > 0:
            g, v = torch.clamp(g, max=case["clamp"]), torch.clamp(v, -case["clamp"], case["clamp"])
        y = _quantised64(g * torch.sigmoid(g) * v) @ _values64(s["down"][0][e], s["down"][1][e]).t().contiguous()
        out.index_add_(0, tok, w[tok, slot].unsqueeze(-1) * y)
    return out, ids.to(torch.int32), w
