"""Plain definitions, in 64 bits unless the definition itself says fp32, of the context-free operators: routing with
groups, the stable pair sort, microscaled 4-bit matrices (codes, scales, tile layout), their product, and the combine.
numpy only; nothing here comes from the library."""
from __future__ import annotations

import numpy as np

BLOCK = {0: 32, 1: 16}  # MOE_MX_E8M0, MOE_MX_E4M3
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
# every non-negative e4m3 number, by its byte (127 is NaN)
E4M3 = np.array([(b & 7) / 8 * 2.0 ** -6 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7) for b in range(127)])


def route(logits, bias, k, G, top_groups, best, sigmoid, renorm, scale):
    """idx int32 [T, k], w fp64 [T, k]."""
    T, E = logits.shape
    idx, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    big = float(np.finfo(np.float32).max)
    for t in range(T):
        l = logits[t].astype(np.float64)
        there = l > -np.inf
        if bias is not None:
            there &= np.asarray(bias, np.float64) > -np.inf
        if not there.any():
            continue
        l = np.where(there, np.minimum(l, big), -np.inf)
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-l)) if sigmoid else np.exp(l - l.max()) / np.exp(l - l.max()).sum()
        s = np.where(there, s, 0)
        c = np.where(there, l if bias is None else s + bias, -np.inf)
        allowed = there
        if top_groups < G:
            v = np.where(there, s, -np.inf) if bias is None and best == 2 else c
            score = []
            for g in range(G):
                q = np.sort(v.reshape(G, -1)[g])[::-1]
                q = q[q > -np.inf][:best]
                score.append(q.sum() if q.size else -np.inf)
            kept = np.argsort(-np.array(score), kind="stable")[:top_groups]
            allowed = there & np.isin(np.arange(E) // (E // G), kept)
        order = np.argsort(-np.where(allowed, c, -np.inf), kind="stable")[:k]
        order = order[allowed[order]]
        if not order.size:
            continue
        idx[t, :order.size] = order
        if renorm:
            # the ratio of scores, relative to the largest chosen logit
            ref = l[order].max()
            with np.errstate(over="ignore"):
                r = np.exp(l[order] - ref)
                if sigmoid:
                    r = r / (1 + np.exp(l[order])) if ref <= 0 else s[order]
            w[t, :order.size] = scale * r / r.sum()
        else:
            w[t, :order.size] = scale * s[order]
    return idx, w


def dispatch(idx, E):
    flat = idx.reshape(-1)
    n, k = flat.size, idx.shape[1]
    kept = np.flatnonzero((flat >= 0) & (flat < E))
    order = kept[np.argsort(flat[kept], kind="stable")]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=E))]).astype(np.int32)
    row = np.full(n, -1, np.int32)
    row[order] = np.arange(order.size)
    token, group = np.full(n, -1, np.int32), np.full(n, -1, np.int32)
    token[:order.size], group[:order.size] = order // k, flat[order]
    return offsets, row.reshape(idx.shape), token, group


def nearest_even(table, a):
    """Index of the entry of an ascending table nearest to each a >= 0 (the even index on a tie, the last one above it)."""
    a = np.asarray(a, np.float64)
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def quantise(x, fmt, t=None):
    """x fp32 [rows, cols] -> codes uint8 [rows, C], scale bytes uint8 [rows, C / B], C = cols rounded up to 256.  The
    definition's quotients and the products with the tensor scale t (one per row, or None) are fp32."""
    B, (rows, cols) = BLOCK[fmt], x.shape
    C = -(-cols // 256) * 256
    p = np.zeros((rows, C), np.float32)
    p[:, :cols] = x
    p = p.reshape(rows, -1, B)
    a = np.abs(p).max(2)
    finite = np.isfinite(p).all(2)
    a = np.where(finite, a, 0).astype(np.float32)
    if fmt == 0:
        e = np.where(a > 0, np.frexp(np.where(a > 0, a, 1).astype(np.float64))[1] - 3, -127)
        e = np.maximum(e, -127)
        byte = (e + 127).astype(np.uint8)
        q = p.astype(np.float64) / np.exp2(e.astype(np.float64))[..., None]
    else:
        t = np.ones((rows, 1), np.float32) if t is None else np.asarray(t, np.float32).reshape(rows, 1)
        byte = nearest_even(E4M3, a / (np.float32(6) * t)).astype(np.uint8)
        d = (E4M3[byte].astype(np.float32) * t)[..., None]
        with np.errstate(all="ignore"):
            q = np.where(d > 0, p / np.where(d > 0, d, 1), 0)
    with np.errstate(invalid="ignore"):
        code = nearest_even(E2M1, np.where(finite[..., None], np.abs(q), 0)).astype(np.uint8)
    code |= (np.signbit(q) & finite[..., None]).astype(np.uint8) << 3
    byte = np.where(finite, byte, 255 if fmt == 0 else 127).astype(np.uint8)
    return code.reshape(rows, C), byte


def scale_values(byte, fmt):
    b = byte.astype(np.int64)
    if fmt == 0:
        return np.where(b == 255, np.nan, np.exp2(b - 127.0))
    return np.where(b == 127, np.nan, np.append(E4M3, np.nan)[b])


def values(code, byte, fmt):
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    s = scale_values(byte, fmt)
    return (v.reshape(*s.shape, BLOCK[fmt]) * s[..., None]).reshape(v.shape)


def tile_bytes(fmt):
    return 16384 + 512 * (256 // (4 * BLOCK[fmt]))


def read_tiles(data, row_tile, in_row, cols, fmt):
    """Codes [n, C] and scale bytes [n, C / B] of the rows at (row_tile, in_row) out of raw tile bytes."""
    kt, n, r = -(-cols // 256), len(row_tile), np.asarray(in_row)
    t = data.reshape(-1, kt, tile_bytes(fmt))
    chunk = np.arange(8) ^ (r & 7)[:, None]  # where the 16-byte chunks 0..7 of each row stand
    b = t[:, :, :16384].reshape(-1, kt, 128, 8, 16)[row_tile[:, None], :, r[:, None], chunk]  # [n, 8, kt, 16]
    b = b.transpose(0, 2, 1, 3).reshape(n, kt * 128)
    s = t[:, :, 16384:].reshape(t.shape[0], kt, -1, 32, 4, 4)[row_tile, :, :, r % 32, r // 32]  # [n, kt, atoms, 4]
    return np.stack([b & 15, b >> 4], 2).reshape(n, kt * 256), s.reshape(n, kt * (256 // BLOCK[fmt]))


def write_tiles(codes, scales, row_tile, in_row, tiles, fmt):
    """Raw tile bytes with the given rows; every other byte 0xFF (NaN scales), which no result may depend on."""
    n, kt, r = len(row_tile), codes.shape[1] // 256, np.asarray(in_row)
    atoms = 256 // (4 * BLOCK[fmt])
    c = np.full((tiles, kt, 128, 8, 16), 0xFF, np.uint8)
    s = np.full((tiles, kt, atoms, 32, 4, 4), 0xFF, np.uint8)
    b = (codes[:, 0::2] | codes[:, 1::2] << 4).reshape(n, kt, 8, 16)
    c[row_tile[:, None], :, r[:, None], np.arange(8) ^ (r & 7)[:, None]] = b.transpose(0, 2, 1, 3)
    s[row_tile, :, :, r % 32, r // 32] = scales.reshape(n, kt, atoms, 4)
    return np.concatenate([c.reshape(tiles, kt, -1), s.reshape(tiles, kt, -1)], 2).reshape(-1)


def ragged_place(offsets, group_of_row):
    o = np.asarray(offsets, np.int64)[group_of_row]
    q = np.arange(len(group_of_row)) - o
    return o // 128 + group_of_row + q // 128, q % 128


def uniform_place(groups, rows):
    r = np.arange(groups * rows)
    return r // rows * -(-rows // 128) + r % rows // 128, r % rows % 128
