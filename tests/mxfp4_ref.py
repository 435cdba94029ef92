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
