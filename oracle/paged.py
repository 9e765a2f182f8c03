"""The paged K/V cache, by its definition (numpy, float64).  Test
infrastructure only.

A pool is uint8 [num_pages, page_size, row].  A row holds one position, all kv
heads: bf16 values and 16 zero bytes, or E4M3 codes, one E8M0 scale byte
(2^(byte - 127), 255 NaN) per kv head and zeros to 16 bytes.  Position j of
sequence b is row j % page_size of page table[b, j // page_size].

A written scale is 2^e, e the least integer in [-118, 119] with max |x| <=
448 * 2^e over the finite values of one position and kv head; a code is the
nearest E4M3 value of x / 2^e, ties to the even code, magnitudes above 448
clamped, and NaN for what is not finite.
"""
from __future__ import annotations

import math

import numpy as np

from .reference import _f64, bf16_bits_to_f64, e4m3_bits_to_f64

D = 128
BF16, E4M3 = 0, 1


def row_bytes(kv_type: int, hkv: int) -> int:
    return hkv * D * (2 if kv_type == BF16 else 1) + 16


def e4m3_nearest(x) -> np.ndarray:
    """Codes (uint8) of the nearest E4M3 values of x; ties to the even code,
    |x| > 448 clamped, NaN (0x7F) for what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    vals = e4m3_bits_to_f64(np.arange(127))           # ascending, 0 .. 448
    a = np.minimum(np.where(np.isfinite(x), np.abs(x), 0.0), vals[-1])
    hi = np.searchsorted(vals, a)                     # vals[hi - 1] < a <= vals[hi]
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - vals[lo], vals[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a == vals[hi], hi, code)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def scale_exponent(x) -> np.ndarray:
    """The exponents e of x [..., 128] (float64), by trying each in turn."""
    x = np.asarray(x, dtype=np.float64)
    top = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    e = np.full(top.shape, -118, dtype=np.int64)
    for _ in range(119 + 118):
        e = np.where((top > 448.0 * np.exp2(e.astype(np.float64))) & (e < 119), e + 1, e)
    return e


def make_row(x_bits, kv_type: int) -> np.ndarray:
    """The cache row (uint8) of one token's new values [Hkv, 128] (bf16 bits)."""
    x_bits = np.asarray(x_bits, dtype=np.uint16)
    hkv = x_bits.shape[0]
    if kv_type == BF16:
        return np.concatenate([x_bits.reshape(-1).view(np.uint8), np.zeros(16, np.uint8)])
    x = bf16_bits_to_f64(x_bits)
    e = scale_exponent(x)
    with np.errstate(invalid="ignore"):
        codes = e4m3_nearest(x / np.exp2(e.astype(np.float64))[:, None])
    tail = np.zeros(16, np.uint8)
    tail[:hkv] = e + 127
    return np.concatenate([codes.reshape(-1), tail])


def row_values(rows, kv_type: int) -> np.ndarray:
    """float64 values [..., Hkv, 128] of cache rows [..., row] (uint8)."""
    rows = np.ascontiguousarray(rows)
    if kv_type == BF16:
        v = bf16_bits_to_f64(rows[..., :-16].copy().view(np.uint16))
        return v.reshape(rows.shape[:-1] + ((rows.shape[-1] - 16) // (2 * D), D))
    hkv = (rows.shape[-1] - 16) // D
    v = e4m3_bits_to_f64(rows[..., :hkv * D]).reshape(rows.shape[:-1] + (hkv, D))
    s = rows[..., hkv * D:hkv * D + hkv]
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return v * scale[..., None]


def slots(table, b: int, pos, page_size: int, num_pages: int) -> np.ndarray:
    """Rows (page * page_size + offset) of positions of sequence b, positions
    clamped into the table and pages into the pool, as reads do."""
    pos = np.clip(np.asarray(pos, dtype=np.int64), 0, table.shape[1] * page_size - 1)
    page = np.clip(table[b, pos // page_size].astype(np.int64), 0, num_pages - 1)
    return page * page_size + pos % page_size


def _spans(q_start, kv_len, n: int, capacity: int):
    """(first token, q_len, kv_len) of each sequence."""
    for b in range(len(kv_len)):
        a = min(max(int(q_start[b]), 0), n)
        e = min(max(int(q_start[b + 1]), a), n)
        yield a, e - a, min(max(int(kv_len[b]), 0), capacity)


def paged_write(x_bits, pool, table, q_start, kv_len, kv_type: int) -> np.ndarray:
    """The pool after the new tokens x_bits [N, Hkv, 128] (bf16 bits) of K or V."""
    pool = pool.copy()
    num_pages, page_size, row = pool.shape
    flat = pool.reshape(-1, row)
    capacity = table.shape[1] * page_size
    for b, (a, n, _) in enumerate(_spans(q_start, kv_len, x_bits.shape[0], capacity)):
        for t in range(n):
            pos = int(kv_len[b]) - n + t
            if not 0 <= pos < capacity:
                continue
            page = int(table[b, pos // page_size])
            if 0 <= page < num_pages:
                flat[page * page_size + pos % page_size] = make_row(x_bits[a + t], kv_type)
    return pool


def paged_gather(pool, table, idx, count, kv_type: int) -> np.ndarray:
    """float64 values [B, k, Hkv, 128] of the selected rows; zeros from count on."""
    num_pages, page_size, row = pool.shape
    B, k = idx.shape
    hkv = (row - 16) // (D * (2 if kv_type == BF16 else 1))
    out = np.zeros((B, k, hkv, D))
    for b in range(B):
        c = min(max(int(count[b]), 0), k)
        s = slots(table, b, idx[b, :c], page_size, num_pages)
        out[b, :c] = row_values(pool.reshape(-1, row)[s], kv_type)
    return out


def attend(q, K, V, scale: float | None = None):
    """One query token q [Hq, 128] over rows K, V [n, Hkv, 128] (float64).
    Returns out [Hq, 128], lse [Hq], and what a bound on a rounded evaluation
    needs: sum_j p_j |v_j| [Hq, 128] and max_j scale * sum_i |q_i k_ji| [Hq]."""
    q = _f64(q)
    Hq, n = q.shape[0], K.shape[0]
    out, mag = np.zeros((Hq, D)), np.zeros((Hq, D))
    lse, zabs = np.full(Hq, -np.inf), np.zeros(Hq)
    if scale is None or scale <= 0:
        scale = 1.0 / math.sqrt(D)
    if n == 0:
        return out, lse, mag, zabs
    G = Hq // K.shape[1]
    for h in range(Hq):
        k, v = K[:, h // G], V[:, h // G]
        z = (k @ q[h]) * scale
        m = z.max()
        p = np.exp(z - m)
        out[h] = (p @ v) / p.sum()
        mag[h] = (p @ np.abs(v)) / p.sum()
        lse[h] = m + math.log(p.sum())
        zabs[h] = (np.abs(k) @ np.abs(q[h])).max() * scale
    return out, lse, mag, zabs


def paged_attention(q, pool_k, pool_v, table, q_start, kv_len, kv_type: int, scale: float | None = None):
    """Chunk attention: q [N, Hq, 128]; token t of sequence b sees positions
    0 .. kv_len - q_len + t.  Returns out, lse, mag, zabs as attend(), by
    token, NaN for tokens of no sequence."""
    q = _f64(q)
    N, Hq, _ = q.shape
    num_pages, page_size, row = pool_k.shape
    res = [np.full((N, Hq, D), np.nan), np.full((N, Hq), np.nan), np.full((N, Hq, D), np.nan), np.full((N, Hq), np.nan)]
    for b, (a, n, kv) in enumerate(_spans(q_start, kv_len, N, table.shape[1] * page_size)):
        s = slots(table, b, np.arange(kv), page_size, num_pages)
        K, V = (row_values(p.reshape(-1, row)[s], kv_type) for p in (pool_k, pool_v))
        for t in range(n):
            seen = max(kv - n + t + 1, 0)
            for dst, val in zip(res, attend(q[a + t], K[:seen], V[:seen], scale)):
                dst[a + t] = val
    return res


def paged_sparse_attention(q, pool_k, pool_v, table, idx, count, kv_type: int, scale: float | None = None):
    """One token per sequence over its selected positions; results as attend()."""
    q = _f64(q)
    B, Hq, _ = q.shape
    num_pages, page_size, row = pool_k.shape
    res = [np.zeros((B, Hq, D)), np.zeros((B, Hq)), np.zeros((B, Hq, D)), np.zeros((B, Hq))]
    for b in range(B):
        c = min(max(int(count[b]), 0), idx.shape[1])
        s = slots(table, b, idx[b, :c], page_size, num_pages)
        K, V = (row_values(p.reshape(-1, row)[s], kv_type) for p in (pool_k, pool_v))
        for dst, val in zip(res, attend(q[b], K, V, scale)):
            dst[b] = val
    return res
