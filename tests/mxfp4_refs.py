"""Plain numpy forms, in 64 bits, of the MXFP4 format, its grouped products and
the token permutation."""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """x [rows][cols] -> (codes uint8 [rows][cols/2], scales uint8 [rows][cols/32])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    floor_log2 = np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] - 1, -1000)
    s = np.clip(floor_log2 - 2 + 127, 0, 254)
    a = np.abs(b) / np.ldexp(1.0, s - 127)[..., None]
    # nearest of the eight magnitudes; a tie goes to the even code
    d = np.abs(a[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    near = d == best
    code = np.where((near & (np.arange(8) % 2 == 0)).any(-1),
                    np.argmax(near & (np.arange(8) % 2 == 0), -1), np.argmax(near, -1))
    code = code | np.where(np.signbit(b), 8, 0)
    code = np.where(bad[..., None], 0, code).reshape(x.shape).astype(np.uint8)
    s = np.where(bad, 255, s).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), s


def values(q, s):
    """The values of codes [..., K/2] with scales [..., K/32]."""
    q, s = np.asarray(q), np.asarray(s).astype(np.int64)
    c = np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)
    v = np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, np.where(s == 255, 0, s - 127)))
    return (v.reshape(*s.shape, 32) * scale[..., None]).reshape(*q.shape[:-1], -1)


def product(a, mats, offsets):
    """(y, sum of |terms|) [rows][N]; rows past offsets[-1] stay 0."""
    y = np.zeros((a.shape[0], mats[0].shape[0]))
    t = np.zeros_like(y)
    for e, m in enumerate(mats):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        y[lo:hi] = a[lo:hi] @ m.T
        t[lo:hi] = np.abs(a[lo:hi]) @ np.abs(m).T
    return y, t


def product_bound(K, terms):
    """What f32 sums may be off: a block's 32 products are multiples of one power
    of two with at most 13 bits, so roundings (or truncations, 2^-23) come from
    adding the K / 32 block sums, the four of one instruction among them."""
    return (K / 32 + 4) * 2.0 ** -23 * terms


def interleave(gate, up):
    """[inter][..] gate and up rows in alternating blocks of 16."""
    g = gate.reshape(-1, 16, *gate.shape[1:])
    u = up.reshape(-1, 16, *up.shape[1:])
    return np.stack([g, u], 1).reshape(-1, *gate.shape[1:])


def sort(idx, E):
    """(offsets, perm, inv) of the assignments sorted by expert, in order within one."""
    flat = idx.reshape(-1)
    order = [a for e in range(E) for a in np.nonzero(flat == e)[0]]
    inv = np.full(flat.size, -1, dtype=np.int32)
    inv[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    return offsets.astype(np.int32), np.array(order, dtype=np.int32), inv.reshape(idx.shape)


def by_slot(rows, inv):
    """[T][k][H]: the row of every slot, 0 where it has none."""
    return np.where((inv >= 0)[..., None], rows[np.maximum(inv, 0)], 0.0)
