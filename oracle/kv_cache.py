"""Oracle: the quantised, paged key/value cache (test infrastructure only).

The group min-max quantizer of ``quantizer`` (0539edu.com/news/6111416 §2.1, §4.2) on keys and
values, per token and head, in groups of g consecutive elements: scale = (max - min)/maxq rounded
up to fp16 with the range widened to contain 0, zero = rint(-min/scale), code =
clamp(rint(x/scale) + zero, 0, maxq). A group that holds a NaN or an infinity, or whose scale is
above fp16's range, stores scale NaN, zero 0 and codes 0. Reading back gives scale·(code - zero).
"""

import numpy as np

from . import quantizer


def quantize(x, bits, g):
    """x [n, H, D] -> (codes int64 [n, H, D], scales, zeros fp64 [n, H, D/g])."""
    maxq = 2 ** bits - 1
    x = np.asarray(x, np.float64)
    n, H, D = x.shape
    xg = x.reshape(n, H, D // g, g)
    finite = np.all(np.isfinite(xg), axis=-1)
    safe = np.where(finite[..., None], xg, 0.0)
    with np.errstate(over="ignore"):
        scale, zero = quantizer.group_params(safe.min(-1), safe.max(-1), maxq)
    good = finite & np.isfinite(scale)
    s1 = np.where(good, scale, 1.0)[..., None]
    q = quantizer.quantize(np.where(good[..., None], safe, 0.0), s1, zero[..., None], maxq)
    return (np.where(good[..., None], q, 0).reshape(n, H, D),
            np.where(good, scale, np.nan), np.where(good, zero, 0.0))


def pack(codes, bits):
    """Codes [..., D] -> bytes [..., D*bits/8], the even element in the low nibble."""
    c = codes.astype(np.uint8)
    return c if bits == 8 else (c[..., 0::2] | (c[..., 1::2] << 4))


def unpack(rows, bits):
    if bits == 8:
        return rows.astype(np.int64)
    out = np.empty(rows.shape[:-1] + (2 * rows.shape[-1],), np.int64)
    out[..., 0::2], out[..., 1::2] = rows & 15, rows >> 4
    return out


def write(codes, scales, zeros, K, V, slots, bits):
    """In place on the cache's arrays (codes uint8, scales and zeros fp16 or wider; the layout
    [2, n_pages, page_size, H, ...])."""
    g = (codes.shape[-1] * 8 // bits) // scales.shape[-1]
    n_slots = codes.shape[1] * codes.shape[2]
    flat = [a.reshape((2, n_slots) + a.shape[3:]) for a in (codes, scales, zeros)]
    for plane, x in enumerate((K, V)):
        q, s, z = quantize(x, bits, g)
        for t, slot in enumerate(slots):
            if 0 <= slot < n_slots:
                flat[0][plane, slot] = pack(q[t], bits)
                flat[1][plane, slot], flat[2][plane, slot] = s[t], z[t]


def read(codes, scales, zeros, page_table, cu_lens, bits):
    """(K, V) fp64 [cu_lens[-1] - cu_lens[0], H, D]: every sequence's positions in turn."""
    page_size = codes.shape[2]
    q = unpack(codes, bits)
    D = q.shape[-1]
    g = D // scales.shape[-1]
    s = np.repeat(np.asarray(scales, np.float64), g, axis=-1)
    z = np.repeat(np.asarray(zeros, np.float64), g, axis=-1)
    out = [[], []]
    for b in range(len(cu_lens) - 1):
        for pos in range(int(cu_lens[b + 1]) - int(cu_lens[b])):
            at = (int(page_table[b][pos // page_size]), pos % page_size)
            for plane in (0, 1):
                i = (plane,) + at
                out[plane].append(s[i] * (q[i] - z[i]))
    shape = (0,) + codes.shape[3:4] + (D,)
    return tuple(np.stack(o) if o else np.zeros(shape) for o in out)
