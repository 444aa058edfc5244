"""The paged KV cache in 64 bits: a plain numpy implementation of the formats
and operators that include/fathom.h defines, one row at a time, sharing no
code with the CUDA path.

A cache here is (codes_k, codes_v, bytes_k, bytes_v), numpy arrays
[pages][H][page_tokens][D] (uint16 bf16 patterns, int8, or uint8 e4m3
patterns) and uint8 [pages][H][page_tokens][D/32] (None for bf16).
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32
LOWEST = -100


def e4m3_table() -> np.ndarray:
    """Values of the 256 patterns: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f is NaN."""
    out = np.zeros(256)
    for p in range(256):
        s, e, m = p >> 7, (p >> 3) & 15, p & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        if e == 15 and m == 7:
            v = math.nan
        out[p] = -v if s else v
    return out


_E4M3 = e4m3_table()


def bf16_value(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_bits(x: np.ndarray) -> np.ndarray:
    """Nearest bf16 of finite fp32 values, ties to even."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def encode(row: np.ndarray, fmt: str):
    """Codes and exponent bytes of one row [D] of fp32 values."""
    if fmt == "bf16":
        return bf16_bits(row), None
    x = row.astype(np.float64)
    codes, scale = np.zeros(len(x), np.int64), np.zeros(len(x) // BLOCK, np.uint8)
    for i in range(len(scale)):
        blk = x[BLOCK * i:BLOCK * (i + 1)]
        if not np.all(np.isfinite(blk)):
            scale[i] = 255
            continue
        m = float(np.max(np.abs(blk)))
        e, top = LOWEST, 121 if fmt == "int8" else 7
        if m > 0:
            # the least exponent that keeps the block's largest value inside the codes
            e = min(top, max(LOWEST, math.frexp(m)[1] - 12))
            while e < top and (round(math.ldexp(m, -e)) > 127 if fmt == "int8" else math.ldexp(m, -e) > 464):
                e += 1
        y = np.ldexp(blk, -e)
        if fmt == "int8":
            c = np.clip(np.rint(y), -127, 127).astype(np.int64)
        else:
            c = np.array([_nearest_e4m3(v) for v in y])
        codes[BLOCK * i:BLOCK * (i + 1)] = c
        scale[i] = e + 127
    return (codes.astype(np.int8) if fmt == "int8" else codes.astype(np.uint8)), scale


def _nearest_e4m3(v: float) -> int:
    a = min(abs(v), 448.0)
    best = min(range(0x7F), key=lambda p: (abs(_E4M3[p] - a), p & 1))   # ties to the even pattern
    return best | (0x80 if math.copysign(1.0, v) < 0 else 0)


def decode(codes: np.ndarray, scale, fmt: str) -> np.ndarray:
    """fp64 values of rows [..., D]."""
    if fmt == "bf16":
        return bf16_value(codes)
    x = codes.astype(np.float64) if fmt == "int8" else _E4M3[codes]
    f = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return x * np.repeat(f, BLOCK, -1)


def place(table_row, pages: int, page_tokens: int, pos: int):
    """(page, token) of a position, or None where it names no token."""
    if pos < 0 or pos // page_tokens >= len(table_row):
        return None
    page = int(table_row[pos // page_tokens])
    return (page, pos % page_tokens) if 0 <= page < pages else None


def rows(cu, length, total: int):
    """(row, sequence, position) of the rows of a call."""
    for b in range(len(length)):
        for r in range(int(cu[b]), min(int(cu[b + 1]), total)):
            yield r, b, int(length[b]) - int(cu[b + 1]) + r


def write(cache, fmt: str, k, v, table, cu, length):
    """The cache with rows k, v [rows][H][D] (fp32 values) put in."""
    cache = [None if a is None else a.copy() for a in cache]
    pages, H, page_tokens, _ = cache[0].shape
    for r, b, pos in rows(cu, length, len(k)):
        at = place(table[b], pages, page_tokens, pos)
        if at is None:
            continue
        for h in range(H):
            for s, x in enumerate((k, v)):
                codes, scale = encode(x[r, h], fmt)
                cache[s][at[0], h, at[1]] = codes
                if scale is not None:
                    cache[2 + s][at[0], h, at[1]] = scale
    return cache


def read(cache, fmt: str, table, cu, length, total: int):
    """K and V [H][total][D] of the call's rows; rows of no sequence are NaN."""
    pages, H, page_tokens, D = cache[0].shape
    out = [np.full((H, total, D), np.nan) for _ in range(2)]
    for r, b, pos in rows(cu, length, total):
        at = place(table[b], pages, page_tokens, pos)
        for s in range(2):
            out[s][:, r] = 0 if at is None else decode(
                cache[s][at[0], :, at[1]], None if cache[2 + s] is None else cache[2 + s][at[0], :, at[1]], fmt)
    return out


def _gather(cache, fmt, table_row, positions):
    """(K, V, ok): values [len][H][D] of positions, and which name a token."""
    pages, H, page_tokens, D = cache[0].shape
    at = [place(table_row, pages, page_tokens, int(p)) for p in positions]
    ok = np.array([a is not None for a in at], bool)
    pg = np.array([a[0] if a else 0 for a in at], np.int64)
    tk = np.array([a[1] if a else 0 for a in at], np.int64)
    kv = [decode(cache[s][pg, :, tk], None if cache[2 + s] is None else cache[2 + s][pg, :, tk], fmt) for s in range(2)]
    return kv[0], kv[1], ok


def _softmax_rows(x, seen):
    """Weights of scores x [rows][keys] over the keys seen (rows of none: zeros)."""
    x = np.where(seen, x, -np.inf)
    top = x.max(-1, keepdims=True, initial=-np.inf)
    p = np.where(seen, np.exp(x - np.where(np.isfinite(top), top, 0)), 0.0)
    total = p.sum(-1, keepdims=True)
    return p / np.where(total > 0, total, 1)


def attend(cache, fmt: str, q, table, cu, length, scale: float, causal: bool = True, max_new=None, max_len=None):
    """out [rows][H*G][D], and what its rounding errors scale with: the sum of |p v| of each value and, per
    (row, head), the largest scale * sum |q k| of a key it sees.  Rows that are not computed are NaN."""
    H = cache[0].shape[1]
    G, D = q.shape[1] // H, q.shape[2]
    out, mag, l1 = np.full(q.shape, np.nan), np.full(q.shape, np.nan), np.zeros(q.shape[:2])
    q = q.astype(np.float64)
    for b in range(len(length)):
        lo, hi, n = int(cu[b]), int(cu[b + 1]), max(0, int(length[b]))
        keys = n if max_len is None else min(n, max_len)
        K, V, ok = _gather(cache, fmt, table[b], range(keys))
        r = np.arange(lo, min(hi, len(q)) if max_new is None else min(hi, lo + max_new, len(q)))
        pos = n - hi + r if length[b] >= 0 else int(length[b]) - hi + r
        seen = ok[None, :] & ((np.arange(keys)[None, :] <= pos[:, None]) if causal else np.ones((len(r), keys), bool))
        for hq in range(H * G):
            keyr, vals = np.where(ok[:, None], K[:, hq // G], 0), np.where(ok[:, None], V[:, hq // G], 0)
            p = _softmax_rows((q[r, hq] @ keyr.T) * scale, seen)
            out[r, hq] = p @ vals
            mag[r, hq] = p @ np.abs(vals)
            l1[r, hq] = np.where(seen, np.abs(scale) * (np.abs(q[r, hq]) @ np.abs(keyr).T), 0).max(-1, initial=0)
    return out, mag, l1


def union_attend(cache, fmt: str, q, table_row, n: int, idx, count, scale: float):
    """out [H][G][D] over each group's listed rows, and its error scales as ``attend`` gives them."""
    out, mag, l1 = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    for h in range(q.shape[0]):
        at = idx[h, :max(0, min(int(count[h]), idx.shape[1]))]
        at = at[(at >= 0) & (at < n)]
        K, V, ok = _gather(cache, fmt, table_row, at)
        x = (q[h].astype(np.float64) @ K[:, h].T) * scale
        p = _softmax_rows(x, np.broadcast_to(ok[None, :], x.shape))
        out[h] = p @ V[:, h]
        mag[h] = p @ np.abs(V[:, h])
        l1[h] = (abs(scale) * (np.abs(q[h]).astype(np.float64) @ np.abs(K[:, h]).T)).max(-1, initial=0)
    return out, mag, l1
