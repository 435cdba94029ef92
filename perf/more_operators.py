"""The 8-bit key/value cache and the attention over it: what is measured, and their plain forms.

Three operators of an engine that keeps its attention cache in pages of int8
codes with one fp32 scale for each block of tokens and head: writing new tokens
into the cache (quantised, older tokens of a block requantised where its scale
grows), reading tokens back, and causal attention over the cache, for single
tokens and for prompts.  `run` computes them in elementary torch operations, or,
where `own` is true, through the framework's calls.

Codes are compared as the values that they stand for, so a write is measured
together with the read of the blocks that it touched.  The cache's arrays are
the same on both sides:
  k codes  [page][head][token / 16][dim / 16][token % 16][dim % 16]
  v codes  [page][head][token / 4][dim][token % 4]
  scales   [page][head][token / block]
(tokens of a page), held as [pages][heads][page size][dims] and
[pages][heads][blocks].
"""
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZES = {"fp32": 4, "bf16": 2, "fp16": 2}


# ---- cases ---------------------------------------------------------------
# seqs sequences with up to `new` new tokens each and up to `len` tokens in all (ragged: sizes spread below these, the first
# sequence has the largest), the last `empty` of them without any cached token; hq query heads on hkv heads of d values.

def _case(op, seqs, new, length, hq, hkv, d, dtype="bf16", page=64, block=16, ragged=False, empty=0, window=0, sinks=False, lse=False, fused=False):
    return {"op": op, "seqs": seqs, "new": new, "len": length, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "page": page, "block": block, "ragged": ragged,
            "empty": empty, "window": window, "sinks": sinks, "lse": lse, "fused": fused}


def listed():
    return [
        # A decode step's new tokens, eight sequences in the middle of their blocks: the launches are the cost.
        {"name": "write_decode_8", **_case("write", 8, 1, 1000, 32, 8, 128, ragged=True)},
        # Several ragged prompts appended behind earlier ones, rows cut out of a fused projection, larger blocks.
        {"name": "write_ragged_9x700", **_case("write", 9, 700, 900, 16, 4, 64, dtype="fp16", page=128, block=64, ragged=True, fused=True)},
        # A long prompt written at once.
        {"name": "write_prompt_16384", **_case("write", 1, 16384, 16384, 32, 8, 128)},
        # One sequence of odd length read back at full precision (a cache that moves to another place).
        {"name": "read_1x1001", **_case("read", 1, 1001, 1001, 8, 2, 256, dtype="fp32", page=32, block=32)},
        # A batch of whole sequences read back.
        {"name": "read_16x4000", **_case("read", 16, 4000, 4000, 32, 8, 128, page=256, ragged=True)},
        # One sequence decoding: the smallest attention call.
        {"name": "decode_1x2000", **_case("attn", 1, 1, 2000, 32, 8, 128)},
        # A full batch decoding, lengths spread, four slots of the batch unused.
        {"name": "decode_64x8192", **_case("attn", 64, 1, 8192, 32, 8, 128, ragged=True, empty=4)},
        # One very long sequence: the token axis is all there is to spread over the card.
        {"name": "decode_1x131072", **_case("attn", 1, 1, 131072, 32, 8, 128, page=256, block=32, lse=True)},
        # The engine's own attention layout: 64 query heads of 512 values on one head, a few sequences, with sinks.
        {"name": "decode_mqa_12x6000", **_case("attn", 12, 1, 6000, 64, 1, 512, page=128, block=32, ragged=True, sinks=True)},
        # Drafted tokens verified: a few new tokens a sequence, odd head counts, a window, two unused slots.
        {"name": "verify_13x5_window", **_case("attn", 13, 5, 3000, 15, 5, 64, dtype="fp16", page=32, ragged=True, empty=2, window=1000, sinks=True, lse=True)},
        # Chunks of prompts over what is cached already, at full precision.
        {"name": "chunk_4x600_fp32", **_case("attn", 4, 600, 2500, 8, 2, 192, dtype="fp32", page=64, block=64, ragged=True, fused=True)},
        # A long prompt: bound by the matrix cores.
        {"name": "prompt_8192", **_case("attn", 1, 8192, 8192, 32, 8, 128)},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("write", "read", "attn", "attn"))
    d = rng.choice((64, 128, 128, 192, 256, 512))
    hkv = _log_int(rng, 1, 8 if d < 512 else 2)
    g = _log_int(rng, 1, 8) if hkv > 1 else _log_int(rng, 1, 64)
    page = rng.choice((16, 32, 64, 128, 256))
    block = rng.choice([b for b in (16, 32, 64, 128) if b <= page])
    common = {"dtype": rng.choice(("bf16", "fp16", "bf16", "fp32")), "page": page, "block": block, "ragged": rng.random() < 0.7}
    if op != "attn":
        total = _log_int(rng, 1, min(40000, 2 ** 25 // (hkv * d)))  # new tokens in all
        seqs = _log_int(rng, 1, min(32, total))
        new = max(1, total // seqs)
        length = new if op == "read" else new + rng.randint(0, 200)
        return _case(op, seqs, new, length, hkv * g, hkv, d, fused=rng.random() < 0.3, **common)
    form = rng.choice(("decode", "verify", "prompt"))
    if form == "prompt":
        new = _log_int(rng, 32, 4096)
        length = new + rng.choice((0, _log_int(rng, 1, 4000)))
        seqs = rng.randint(1, 4)
    else:
        new = 1 if form == "decode" else rng.randint(2, 8)
        length = _log_int(rng, 64, 65536)
        seqs = _log_int(rng, 1, 64)
    # no more than the largest listed cases: scores, codes
    while seqs > 1 and (seqs * new * hkv * g * length > 2 ** 31 or seqs * length * hkv * d > 2 ** 28):
        seqs //= 2
    while new * hkv * g * length > 2 ** 31 or length * hkv * d > 2 ** 28:
        length = max(length // 2, 32)
        new = min(new, length)
    return _case("attn", seqs, new, length, hkv * g, hkv, d, fused=rng.random() < 0.3, empty=rng.choice((0, seqs // 4)), window=rng.choice((0, 0, 128, 1000)),
                 sinks=rng.random() < 0.3, lse=rng.random() < 0.3, **common)


def _sizes(case):
    """(new tokens, length) of each sequence, by the case alone."""
    rng = random.Random("%d %d %d" % (case["seqs"], case["new"], case["len"]))
    got = []
    for s in range(case["seqs"]):
        new, length = case["new"], case["len"]
        if case["ragged"] and s:
            new = rng.randint(max(1, new // 8), new)
            length = new if case["op"] == "read" else max(new, rng.randint(max(1, length // 4), length))
        if s >= case["seqs"] - case["empty"]:
            new, length = min(new, 1), 0
        got.append((new, length))
    return got


def work(case):
    sizes, e, h, d = _sizes(case), SIZES[case["dtype"]], case["hkv"], case["d"]
    n = sum(new for new, _ in sizes)
    scale = 4 / case["block"]
    if case["op"] == "write":
        # the new rows once, their codes once, the values read back once
        return {"bytes": int(2 * n * h * (d * (e + 1) + scale) + 2 * e * d * h * sum(b - a for a, b in _touched(case))), "flops": 8 * n * h * d}
    if case["op"] == "read":
        return {"bytes": int(2 * n * h * (d * (1 + e) + scale)), "flops": 2 * n * h * d}
    live = pairs = 0
    for new, length in sizes:
        for p in (range(length - new, length) if length else ()):
            pairs += p + 1 if not case["window"] else min(p + 1, case["window"])
        live += length if not case["window"] else min(length, new + case["window"] - 1)
    return {"bytes": int(2 * live * h * (d + scale) + 2 * n * case["hq"] * d * e), "flops": 4 * d * case["hq"] * pairs}


def _touched(case):
    """Each sequence's tokens [from, to) in the blocks that its new tokens fall into."""
    return [((length - new) // case["block"] * case["block"], length) for new, length in _sizes(case)]


# ---- inputs --------------------------------------------------------------

def _rows(shape, g):
    """N(0, 1) with 1% of each head's channels eight times larger, as keys have."""
    x = torch.randn(shape, generator=g, device="cuda")
    return x * (1.0 + 7.0 * (torch.rand(shape[-2:], generator=g, device="cuda") < 0.01))


def _cached(pages, case, g, tiles):
    """(codes, scales) of a pool of pages full of tokens, some pages at a time."""
    h, p, d, b = case["hkv"], case["page"], case["d"], case["block"]
    codes = torch.empty((pages, h, p, d), dtype=torch.int8, device="cuda")
    scales = torch.empty((pages, h, p // b), device="cuda")
    step = max(1, (1 << 26) // (h * p * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = _rows((n, p // b, b, h, d), g).permute(0, 3, 1, 2, 4)
        s = x.abs().amax((-1, -2)) / 127.0
        q = torch.round(x / s[..., None, None]).to(torch.int8).reshape(n, h, p, d)
        codes[i:i + n], scales[i:i + n] = tiles(q), s
    return codes, scales


def _k_tiles(q):
    n, h, p, d = q.shape
    return q.view(n, h, p // 16, 16, d // 16, 16).transpose(3, 4).reshape(n, h, p, d)


def _v_tiles(q):
    n, h, p, d = q.shape
    return q.view(n, h, p // 4, 4, d).transpose(3, 4).reshape(n, h, p, d)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    sizes = _sizes(case)
    h, d, p = case["hkv"], case["d"], case["page"]
    used = [-(-length // p) for _, length in sizes]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(sizes), max(used) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u
    k, ks = _cached(pages, case, g, _k_tiles)
    v, vs = _cached(pages, case, g, _v_tiles)

    def starts_of(counts):
        return torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")

    n = sum(new for new, _ in sizes)
    s = {"case": case, "k": k, "ks": ks, "v": v, "vs": vs, "table": table, "n": n, "starts": starts_of([new for new, _ in sizes]),
         "lens": torch.tensor([length for _, length in sizes], dtype=torch.int32, device="cuda")}
    if case["op"] == "write":
        spans = [b - a for a, b in _touched(case)]
        s["back"], s["n_back"] = starts_of(spans), sum(spans)
    if case["op"] != "read":
        # the step's rows: queries, keys and values beside each other where one projection makes them
        width = (case["hq"] + 2 * h) if case["fused"] else (case["hq"] if case["op"] == "attn" else 2 * h)
        rows = _rows((n, width, d), g).to(DTYPES[case["dtype"]])
        if case["op"] == "attn":
            s["q"] = rows[:, :case["hq"]]
        elif case["fused"]:
            s["new_k"], s["new_v"] = rows[:, case["hq"]:case["hq"] + h], rows[:, case["hq"] + h:]
        else:
            s["new_k"], s["new_v"] = rows[:, :h].contiguous(), rows[:, h:].contiguous()
    s["sinks"] = torch.randn((case["hq"],), generator=g, device="cuda") if case["sinks"] else None
    if own:
        import q8_quantized_matmul_amd as q8
        most = max(new for new, _ in sizes)
        # the cache and the step's batch, as a program keeps them
        s["cache"] = q8.Kv8Cache(k, v, ks, vs)
        s["batch"] = q8.Kv8Batch(table, s["lens"], starts=None if n == len(sizes) and most == 1 else s["starts"], n_tok=n, max_new=most, max_len=case["len"])
        if case["op"] == "write":
            s["back_batch"] = q8.Kv8Batch(table, s["lens"], starts=s["back"], n_tok=s["n_back"], max_new=max(spans), max_len=case["len"])
        if case["op"] == "attn":
            s["workspace"] = q8.kv8_attention_workspace(s["cache"], s["batch"], case["hq"])
            s["lse"] = torch.empty((n, case["hq"]), device="cuda") if case["lse"] else None
    return s


# ---- the plain forms -----------------------------------------------------

def _k_rows(c):
    """Tiled codes [..., heads, page, d] of whole pages as [..., page, heads, d]."""
    lead, (h, p, d) = c.shape[:-3], c.shape[-3:]
    return c.view(*lead, h, p // 16, d // 16, 16, 16).transpose(-3, -2).reshape(*lead, h, p, d).transpose(-3, -2)


def _v_rows(c):
    lead, (h, p, d) = c.shape[:-3], c.shape[-3:]
    return c.view(*lead, h, p // 4, d, 4).transpose(-2, -1).reshape(*lead, h, p, d).transpose(-3, -2)


def _places(s, starts, n):
    """(sequence, position) of each token of a ragged batch."""
    tok = torch.arange(n, device="cuda")
    seq = torch.searchsorted(starts[1:].contiguous(), tok, right=True)
    return seq, s["lens"].long()[seq] - starts.long()[seq + 1] + tok


def _write(s, codes, scales, rows_of, tiles, x):
    c = s["case"]
    p, b = c["page"], c["block"]
    pages, h, _, d = codes.shape
    seq, pos = _places(s, s["starts"], s["n"])
    slot = s["table"].long()[seq, pos // p] * p + pos % p  # of the pool
    blk = slot // b
    x = x.float()
    blocks = pages * p // b
    amax = torch.zeros((blocks, h), device="cuda").index_reduce_(0, blk, x.abs().amax(-1), "amax")
    old = scales.transpose(1, 2).reshape(-1, h)
    # blocks whose first token is new take nothing over; the others keep their older tokens, under a scale that only grows
    touched = torch.zeros((blocks, 1), device="cuda").index_fill_(0, blk, 1.0) > 0
    fresh = torch.zeros(blocks, device="cuda").index_reduce_(0, blk, (pos % b == 0).float(), "amax")[:, None] > 0
    scale = torch.where(touched, torch.maximum(torch.where(fresh, 0.0, old), amax / 127.0), old)
    q = rows_of(codes).reshape(pages * p, h, d)
    grown = (touched & ~fresh & (scale > old)).repeat_interleave(b, 0)[..., None]
    over, under = (t.double().repeat_interleave(b, 0)[..., None] for t in (old, torch.where(scale > 0, scale, 1.0)))
    q = torch.where(grown, torch.round(q.double() * over / under).to(torch.int8), q)
    new = scale[blk].double()[..., None]
    q[slot] = torch.where(new > 0, torch.round(x.double() / new), 0.0).clamp(-127, 127).to(torch.int8)
    codes.copy_(tiles(q.view(pages, p, h, d).transpose(1, 2)))
    scales.copy_(scale.view(pages, p // b, h).transpose(1, 2))


def _read(s, codes, scales, rows_of, starts, n, dtype):
    c = s["case"]
    p, b = c["page"], c["block"]
    pages, h, _, d = codes.shape
    seq, pos = _places(s, starts, n)
    slot = s["table"].long()[seq, pos // p] * p + pos % p
    q = rows_of(codes).reshape(pages * p, h, d)[slot]
    return (q.float() * scales.transpose(1, 2).reshape(-1, h)[slot // b][..., None]).to(dtype)


def _attention(s):
    c = s["case"]
    p, b, h, d = c["page"], c["block"], c["hkv"], c["d"]
    g, n_seq, most = c["hq"] // h, c["seqs"], c["new"]
    table = s["table"].long().clamp(min=0)

    def gather(codes, scales, rows_of):  # [sequence * head, length, d]
        x = rows_of(codes[table]).float().reshape(n_seq, -1, b, h, d) * scales[table].transpose(2, 3).reshape(n_seq, -1, 1, h, 1)
        return x.reshape(n_seq, -1, h, d).transpose(1, 2).reshape(n_seq * h, -1, d)

    seq, pos = _places(s, s["starts"], s["n"])
    row = torch.arange(s["n"], device="cuda") - s["starts"].long()[seq]
    q = torch.zeros((n_seq, most, h, g, d), device="cuda")
    q[seq, row] = s["q"].float().view(-1, h, g, d)
    at = torch.full((n_seq, most), -1, device="cuda")
    at[seq, row] = pos
    z = torch.bmm(q.permute(0, 2, 1, 3, 4).reshape(n_seq * h, most * g, d), gather(s["k"], s["ks"], _k_rows).transpose(1, 2)) * (1.0 / math.sqrt(d))
    z = z.view(n_seq, h, most, g, -1)
    j = torch.arange(z.shape[-1], device="cuda")
    live = j <= at[..., None]
    if c["window"]:
        live &= j > at[..., None] - c["window"]
    z = torch.where(live[:, None, :, None], z, -math.inf)
    top = z.amax(-1, keepdim=True)
    sink = None
    if c["sinks"]:
        sink = s["sinks"].view(1, h, 1, g, 1)
        top = torch.maximum(top, sink)
    top = torch.where(top > -math.inf, top, 0.0)
    w = torch.exp(z - top)
    total = w.sum(-1, keepdim=True)
    if c["sinks"]:
        total = total + torch.exp(sink - top)
    out = torch.bmm(w.view(n_seq * h, most * g, -1), gather(s["v"], s["vs"], _v_rows)).view(n_seq, h, most, g, d)
    out = out / torch.where(total > 0, total, 1.0)
    out = out.permute(0, 2, 1, 3, 4).reshape(n_seq, most, c["hq"], d)[seq, row].to(DTYPES[c["dtype"]])
    if not c["lse"]:
        return out
    return out, (top + torch.log(total)).permute(0, 2, 1, 3, 4).reshape(n_seq, most, c["hq"])[seq, row]


def run(s):
    c = s["case"]
    dtype = DTYPES[c["dtype"]]
    if own:
        import q8_quantized_matmul_amd as q8
        if c["op"] == "write":
            q8.kv8_write(s["cache"], s["batch"], s["new_k"], s["new_v"])
            return q8.kv8_read(s["cache"], s["back_batch"], dtype)
        if c["op"] == "read":
            return q8.kv8_read(s["cache"], s["batch"], dtype)
        out = q8.kv8_attention(s["cache"], s["batch"], s["q"], window=c["window"], sinks=s["sinks"], lse=s["lse"], workspace=s["workspace"])
        return (out, s["lse"]) if c["lse"] else out
    if c["op"] == "write":
        _write(s, s["k"], s["ks"], _k_rows, _k_tiles, s["new_k"])
        _write(s, s["v"], s["vs"], _v_rows, _v_tiles, s["new_v"])
        return _read(s, s["k"], s["ks"], _k_rows, s["back"], s["n_back"], dtype), _read(s, s["v"], s["vs"], _v_rows, s["back"], s["n_back"], dtype)
    if c["op"] == "read":
        return _read(s, s["k"], s["ks"], _k_rows, s["starts"], s["n"], dtype), _read(s, s["v"], s["vs"], _v_rows, s["starts"], s["n"], dtype)
    return _attention(s)


# ---- the definition in 64 bits -------------------------------------------

def _sequence(s, i, length, what):
    """(codes, scales by token) of one sequence's first `length` tokens, in doubles: [length, heads, d] and [length, heads]."""
    c = s["case"]
    p, b, h, d = c["page"], c["block"], c["hkv"], c["d"]
    pages = s["table"][i, :-(-length // p)].long()
    codes = s[what][pages].double()
    if what == "k":
        codes = codes.view(-1, h, p // 16, d // 16, 16, 16).permute(0, 2, 4, 1, 3, 5).reshape(-1, h, d)
    else:
        codes = codes.view(-1, h, p // 4, d, 4).permute(0, 2, 4, 1, 3).reshape(-1, h, d)
    scales = s[what + "s"][pages].double().permute(0, 2, 1).reshape(-1, h).repeat_interleave(b, 0)
    return codes[:length], scales[:length]


def _written64(s, what):
    """The touched blocks' values after the write, a sequence at a time."""
    c, got = s["case"], []
    b, at = c["block"], 0
    for i, (new, length) in enumerate(_sizes(c)):
        first = (length - new) // b * b
        older = length - new - first  # tokens before the new ones in their first block
        codes, scales = (t[first:] for t in _sequence(s, i, length, what))
        x = s["new_" + what][at:at + new].double()
        at += new
        x = torch.cat((codes[:older] * scales[:older, :, None], x))
        pad = -len(x) % b
        blocks = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(-1, b, *x.shape[1:])
        is_new = torch.ones(len(x) + pad, device="cuda", dtype=torch.float64)
        is_new[:older] = 0.0
        step = (blocks * is_new.view(-1, b, 1, 1)).abs().amax((1, 3)).div(127.0).float().double()  # a scale is stored in 32 bits
        if older:
            step[0] = torch.maximum(step[0], scales[0])
        step = step.repeat_interleave(b, 0)[:len(x), :, None]
        got.append(torch.where(step > 0, torch.round(x / torch.where(step > 0, step, 1.0)), 0.0) * step)
    return torch.cat(got)


def _attended64(s):
    c, out, lse, at = s["case"], [], [], 0
    h, d = c["hkv"], c["d"]
    g = c["hq"] // h
    for i, (new, length) in enumerate(_sizes(c)):
        q = s["q"][at:at + new].double().reshape(new, h, g, d)
        at += new
        o = torch.zeros((new, h, g, d), dtype=torch.float64, device="cuda")
        e = torch.full((new, h, g), -math.inf, dtype=torch.float64, device="cuda")
        pos = torch.arange(length - new, length, device="cuda")
        j = torch.arange(length, device="cuda")
        dead = (j > pos[:, None]) | ((j <= pos[:, None] - c["window"]) if c["window"] else False)
        if length:
            k, v = ((a * b[..., None]) for a, b in (_sequence(s, i, length, w) for w in "kv"))
        for head in range(h):  # a head at a time
            sink = s["sinks"].double()[head * g:(head + 1) * g] if c["sinks"] else None
            if not length:
                e[:, head] = e[:, head] if sink is None else sink
                continue
            z = (q[:, head].reshape(new * g, d) @ k[:, head].t().contiguous()).view(new, g, length) / math.sqrt(d)
            z = z.masked_fill(dead[:, None], -math.inf)
            e[:, head] = torch.logsumexp(z, -1) if sink is None else torch.logaddexp(torch.logsumexp(z, -1), sink.expand(new, g))
            o[:, head] = (torch.exp(z - e[:, head, :, None]).view(new * g, length) @ v[:, head].contiguous()).view(new, g, d)
        out.append(o.view(new, h * g, d))
        lse.append(e.view(new, h * g))
    return (torch.cat(out), torch.cat(lse)) if c["lse"] else torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        return _written64(s, "k"), _written64(s, "v")
    if case["op"] == "read":
        got = []
        for what in "kv":
            parts = [(a * b[..., None])[length - new:] for new, length, (a, b) in ((n, m, _sequence(s, i, m, what)) for i, (n, m) in enumerate(_sizes(case)))]
            got.append(torch.cat(parts))
        return tuple(got)
    return _attended64(s)
