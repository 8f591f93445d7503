"""Plain numpy forms, in 64 bits, of the FP8 format (e4m3 codes, a scale for each block of 128), its products and
their gradients, and of routing with groups."""
from __future__ import annotations

import numpy as np

BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def _decode():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 512, np.ldexp(1 + m / 8, e - 7))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


CODES = _decode()                                # the value of every code
_POSITIVE = CODES[:127]


def encode(x):
    """x, at most 448 in size, to the nearest code, a tie to the even one."""
    a = np.abs(x)
    hi = np.searchsorted(_POSITIVE, a).clip(0, 126)
    lo = (hi - 1).clip(0)
    dh, dl = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def scale_code(top):
    """c where 2^(c - 127) is the smallest power of two, c >= 1, that brings `top` to 448 or below."""
    top = np.asarray(top, dtype=np.float64)
    m, e = np.frexp(np.where(np.isfinite(top), top, 1.0) / 448.0)
    e = np.where(m == 0.5, e - 1, e)
    return np.where(np.isfinite(top), np.where(top == 0, 1, np.maximum(e + 127, 1)), 255)


def scale_value(code):
    return np.where(code == 255, np.nan, np.ldexp(1.0, np.where(code == 255, 0, code - 127)))


def _quantize(b, axes):
    """Blocks b (their axes `axes`) -> (codes, scale codes)."""
    bad = ~np.isfinite(b).all(axes, keepdims=True)
    top = np.abs(np.where(bad, 0.0, b)).max(axes, keepdims=True)
    code = np.where(bad, 255, scale_code(top))
    q = encode(np.where(bad, 0.0, b) / np.where(bad, 1.0, scale_value(code)))
    return np.where(bad, 0, q).astype(np.uint8), code


def _pad(x, rows=False):
    return np.pad(x, ((0, -x.shape[0] % BLOCK if rows else 0), (0, -x.shape[1] % BLOCK)))


def quantize_rows(x):
    """x [rows][cols] -> (codes [rows][cols], scale codes [rows][blocks])."""
    x = np.asarray(x, dtype=np.float64)
    q, s = _quantize(_pad(x).reshape(x.shape[0], -1, BLOCK), (2,))
    return q.reshape(x.shape[0], -1)[:, :x.shape[1]], s[..., 0]


def quantize_matrix(x):
    x = np.asarray(x, dtype=np.float64)
    p = _pad(x, True)
    b = p.reshape(p.shape[0] // BLOCK, BLOCK, -1, BLOCK)
    q, s = _quantize(b, (1, 3))
    return q.reshape(p.shape)[:x.shape[0], :x.shape[1]], s[:, 0, :, 0]


def quantize_columns(x, offsets):
    """(codes [blocks][cols][128], scale codes [blocks][cols]) of the experts' rows, as many blocks as they fill."""
    x = np.asarray(x, dtype=np.float64)
    codes, scales = [np.zeros((0, x.shape[1], BLOCK), np.uint8)], [np.zeros((0, x.shape[1]), np.int64)]
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        if hi > lo:
            q, s = quantize_rows(np.pad(x[lo:hi], ((0, -(hi - lo) % BLOCK), (0, 0))).T)
            codes.append(q.reshape(x.shape[1], -1, BLOCK).transpose(1, 0, 2))
            scales.append(s.T)
    return np.concatenate(codes), np.concatenate(scales)


def column_values(q, s):
    """The values of such blocks, [cols][rows]."""
    return (CODES[q] * scale_value(s)[..., None]).transpose(1, 0, 2).reshape(q.shape[1], -1)


def values(q, s, block_rows=1):
    """The values of codes [rows][cols] with scale values for 128 columns of block_rows rows."""
    v = CODES[q]
    s = np.repeat(np.asarray(s, dtype=np.float64), BLOCK, 1)[:, :v.shape[1]]
    return v * (s if block_rows == 1 else np.repeat(s, BLOCK, 0)[:v.shape[0]])


def product(a, mats, offsets):
    """(y, sum of |terms|) [rows][N]; rows outside the offsets are 0."""
    y = np.zeros((a.shape[0], mats[0].shape[0]))
    t = np.zeros_like(y)
    for e, m in enumerate(mats):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        y[lo:hi] = a[lo:hi] @ m.T
        t[lo:hi] = np.abs(a[lo:hi]) @ np.abs(m).T
    return y, t


def product_bound(K, terms, exact):
    """What a product's sums may be off. exact (f32 results): products are exact, each of the K + 2 K / 128
    additions and scalings loses less than 2^-23 of a partial sum. Otherwise also what the FP8 instruction
    cuts off of 8 products at a time: less than 2^-13 of the largest from each."""
    sums = (K + 2 * blocks(K) + 4) * 2.0 ** -23
    return (sums if exact else sums + 2.0 ** -10) * terms


def norm_bound(K, exact):
    """The same for the 2-norm of all errors, which are of either sign: sqrt(K) of them of 2^-24 to 2^-22 of the
    result, and the cut-off products' 1.5e-5 with room."""
    return np.sqrt(K) * 2.0 ** -22 + (0.0 if exact else 2.0 ** -12)


def silu(g):
    return g / (1 + np.exp(-g))


# ------------------------------------------------------------ routing
def scores(logits, kind):
    l = np.asarray(logits, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-l))
        top = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(1, keepdims=True)
    return np.where(total == 0, 0.0, e / np.where(total == 0, 1.0, total))


def route(logits, bias, k, kind, groups, kept, group_top, norm, scale):
    """(idx, w, scores rounded to f32), token by token."""
    T, E = logits.shape
    s = scores(logits, kind).astype(np.float32)
    b = np.zeros(E, np.float32) if bias is None else np.asarray(bias, np.float32)
    idx, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    size = E // groups
    for t in range(T):
        key = [np.float32(-np.inf) if np.isneginf(logits[t, e]) or np.isneginf(b[e]) else np.float32(s[t, e] + b[e])
               for e in range(E)]
        value = []
        for j in range(groups):
            best = sorted((v for v in key[j * size:(j + 1) * size] if v > -np.inf), reverse=True)[:group_top]
            value.append(np.float32(-np.inf) if not best else best[0] if len(best) == 1 else np.float32(best[0] + best[1]))
        order = sorted((j for j in range(groups) if value[j] > -np.inf), key=lambda j: (-value[j], j))[:kept]
        left = [e for e in range(E) if e // size in order and key[e] > -np.inf]
        picks = sorted(left, key=lambda e: (-key[e], e))[:k]
        idx[t, :len(picks)] = picks
        got = s[t, picks].astype(np.float64)
        total = got.sum()
        w[t, :len(picks)] = scale * (got if not norm else got / total if total > 0 else np.full(len(picks), 1 / max(1, len(picks))))
    return idx, w, s


def weights(logits, idx, kind, norm, scale):
    """The weights alone, in 64 bits, for given choices: the function that the gradient is of."""
    s = scores(logits, kind)
    got = np.where(idx >= 0, np.take_along_axis(s, np.maximum(idx, 0), 1), 0.0)
    total = got.sum(1, keepdims=True)
    return scale * (np.where(total > 0, got / np.where(total > 0, total, 1.0), 0.0) if norm else got)


def route_grad(w_grad, logits, idx, kind, norm, scale, scores_grad=None):
    s = scores(logits, kind)
    used = idx >= 0
    at = np.maximum(idx, 0)
    got = np.where(used, np.take_along_axis(s, at, 1), 0.0)
    g = np.where(used, scale * np.asarray(w_grad, np.float64), 0.0)
    if norm:
        total = got.sum(1, keepdims=True)
        safe = np.where(total > 0, total, 1.0)
        g = np.where(used & (total > 0), (g - (g * got).sum(1, keepdims=True) / safe) / safe, 0.0)
    d = np.zeros_like(s) if scores_grad is None else np.asarray(scores_grad, np.float64).copy()
    for j in range(idx.shape[1]):
        np.add.at(d, (np.arange(len(d)), at[:, j]), np.where(used[:, j], g[:, j], 0.0))
    if kind == "sigmoid":
        return d * s * (1 - s)
    return s * (d - (d * s).sum(1, keepdims=True))
