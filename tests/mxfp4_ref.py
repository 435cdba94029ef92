"""Plain 64-bit forms of the MXFP4 operators, for the tests: numpy on the CPU,
from the definitions, sharing no code with the library."""
import numpy as np
import torch

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EVEN = np.arange(8) % 2 == 0


def quantize(x):
    """(codes [rows][k/2], scales [rows][k/32]) of float64 rows."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    b = x.reshape(rows, k // 32, 32)
    finite = np.isfinite(b).all(-1)
    amax = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1), 1.0)
    _, e = np.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    shared = np.where(amax > 0, np.maximum(e - 3, -127), -127)
    scales = np.where(finite, shared + 127, 255).astype(np.uint8)
    a = np.abs(np.where(finite[..., None], b, 0.0)) / np.exp2(shared.astype(np.float64))[..., None]
    a = np.minimum(a, 6.0)
    # The nearest magnitude; of two equally near ones the even code.
    dist = np.abs(a[..., None] - MAGNITUDES)
    best = dist.min(-1, keepdims=True)
    code = np.where((dist == best) & EVEN, np.arange(8), 99).min(-1)
    only_odd = code == 99
    code = np.where(only_odd, dist.argmin(-1), code)
    code = (code + 8 * (np.signbit(b) & finite[..., None])).astype(np.uint8)
    code = code.reshape(rows, k // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), scales


def values(codes, scales):
    """float64 values [..., k] of codes [..., k/2] and scales [..., k/32]."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    nib = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1, 32)
    v = MAGNITUDES[nib & 7] * np.where(nib >= 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return (v * s[..., None]).reshape(*codes.shape[:-1], -1)


def random_matrix(rng, shape, lo=116, hi=126):
    """Uniform codes and scale bytes in [lo, hi] for a matrix [..., k]."""
    codes = rng.integers(0, 256, (*shape[:-1], shape[-1] // 2), dtype=np.uint8)
    scales = rng.integers(lo, hi + 1, (*shape[:-1], shape[-1] // 32)).astype(np.uint8)
    return codes, scales


def device(q8, m):
    return q8.Mxfp4(*(torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in m))


def host(t):
    """float64 numpy values of a device tensor."""
    return t.detach().cpu().double().numpy()


def route(logits, n_used, bias=None, scoring=0, renormalize=True, scale=1.0):
    """(ids int32, weights float64) of float32 logits [t][e]: 0 softmax, 1 sigmoid,
    2 sqrt(softplus).  Softmax keys are fp32 sums, the others float64."""
    z32 = np.asarray(logits, dtype=np.float32)
    z = z32.astype(np.float64)
    t, e = z.shape
    with np.errstate(all="ignore"):
        if scoring == 0:
            score = z
            key = z if bias is None else (z32 + np.asarray(bias, np.float32)).astype(np.float64)
        else:
            score = 1 / (1 + np.exp(-z)) if scoring == 1 else np.sqrt(np.log1p(np.exp(-np.abs(z))) + np.maximum(z, 0))
            key = score if bias is None else score + np.asarray(bias, np.float64)
        key = np.where(np.isneginf(z), -np.inf, key)
        rank = np.where(np.isnan(key), np.inf, key)
        second = np.where(np.isnan(key), 0, 1)          # NaN before +inf
        ids = np.full((t, n_used), -1, dtype=np.int32)
        w = np.zeros((t, n_used))
        for r in range(t):
            order = sorted(range(e), key=lambda i: (-rank[r, i], second[r, i], i))
            chosen = [i for i in order if not np.isneginf(key[r, i])][:n_used]
            ids[r, :len(chosen)] = chosen
            s = score[r, chosen]
            if scoring == 0 and chosen:
                over = s if renormalize else z[r][~np.isneginf(z[r])]
                m = over.max()
                s, total = np.exp(s - m), np.exp(over - m).sum()
            else:
                total = s.sum() if renormalize else 1.0
            w[r, :len(chosen)] = (s if total == 0 else s / total) * scale
    return ids, w


def _rounded(v, e):
    """v rounded to the e2m1 grid at scale 2^e (float64, elementwise)."""
    a = np.minimum(np.abs(v) / np.exp2(e), 6.0)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return np.copysign(np.rint(a / step) * step, v) * np.exp2(e)


def _requantized(mid, delta):
    """The quantized values of mid [n][k], and how far those of any numbers
    within delta of it may be from them (next to a rounding boundary, or in a
    block whose maximum may lie on either side of a power of two)."""
    b, d = mid.reshape(len(mid), -1, 32), delta.reshape(len(mid), -1, 32)

    def exponent(m):
        _, e = np.frexp(m)
        return np.where(m > 0, np.maximum(e - 3, -127), -127).astype(np.float64)[..., None]
    q = _rounded(b, exponent(np.abs(b).max(-1)))
    low = exponent(np.maximum(np.abs(b) - d, 0.0).max(-1))
    high = exponent((np.abs(b) + d).max(-1))
    off = np.zeros_like(b)
    for e in (low, high):
        for end in (b - d, b + d):
            off = np.maximum(off, np.abs(_rounded(end, e) - q))
    return q.reshape(mid.shape), off.reshape(mid.shape)


def moe_layer(x, logits, gate, up, down, n_used, bias=None, scoring=0, renormalize=True, scale=1.0,
              clamp=0.0, half=0.0):
    """(out, tolerance, ids, weights) of the whole layer in 64 bits, from float64
    x and (codes, scales) matrices [e][n][k].

    The tolerance follows the fp32 roundings through the formula: a product's
    (k / 32 + 8) steps of sum |w x|, carried through silu (|silu'| < 1.1) with
    16 half steps for its own evaluation; mid values that may fall on the other
    side of a rounding boundary; the down product's steps; the weights' roundings
    and one per expert in the sum; `half` for the rounding of the output."""
    step = 2.0 ** -23
    x4 = values(*quantize(x))
    t, d = x4.shape
    f = gate[0].shape[1]
    ids, weights = route(logits, n_used, bias, scoring, renormalize, scale)
    z = np.asarray(logits, np.float64)
    z = z[np.isfinite(z) & (z > -1e30)]
    wrel = ((float(z.max() - z.min()) if z.size else 0.0) + 32) * step / 2
    out, tol, mag = np.zeros((t, d)), np.zeros((t, d)), np.zeros((t, d))
    for e in np.unique(ids[ids >= 0]):
        tok, slot = np.nonzero(ids == e)
        wg, wu, wd = (values(m[0][e], m[1][e]) for m in (gate, up, down))
        g, u = x4[tok] @ wg.T, x4[tok] @ wu.T
        dg, du = ((d / 32 + 8) * step * (np.abs(x4[tok]) @ np.abs(w).T) for w in (wg, wu))
        if clamp > 0:
            g, u = np.minimum(g, clamp), np.clip(u, -clamp, clamp)
        silu = g / (1 + np.exp(-g))
        mid = silu * u
        delta = 1.1 * np.abs(u) * dg + np.abs(silu) * du + 1.1 * dg * du + 8 * step * np.abs(mid)
        q, off = _requantized(mid, delta)
        y = q @ wd.T
        dy = off @ np.abs(wd).T + (f / 32 + 8) * step * ((np.abs(q) + off) @ np.abs(wd).T)
        w = weights[tok, slot][:, None]
        np.add.at(out, tok, w * y)
        np.add.at(tol, tok, np.abs(w) * dy * (1 + wrel))
        np.add.at(mag, tok, np.abs(w * y))
    tol += mag * (wrel + (n_used + 2) * step / 2) + half * np.abs(out) + 1e-30
    return out, tol, ids, weights
