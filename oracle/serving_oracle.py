"""Float64 CPU oracle of the serving operators: 4-bit weights, rotary positions and the 8-bit key/value cache.

TEST INFRASTRUCTURE ONLY, like fusedlin_oracle: plain definitions in float64 NumPy, imported by tests only.

Codes are those of the exact quotient by the stored scale. A float64 quotient of two values of at most 24 significant
bits never rounds onto or across a border between two codes that the exact quotient does not lie on: the border
has at most 9 significant bits, so x - border * scale is a multiple of 2^-32 of the operands' last places, and
the quotient's relative distance from the border is 2^-33 at least, where float64 rounds at 2^-53.
"""
from __future__ import annotations

import numpy as np

KV_TOP = {"int8": 127.0, "e4m3": 448.0}
KV_TINY = 2.0 ** -126


def w4_quantize(W, group, round_scale, least):
    """Codes [N, K] (0 .. 15) and scales [N, K / group] of a weight [N, K]; round_scale rounds to the dtype, whose
    smallest positive value is `least`."""
    W = np.asarray(W, dtype=np.float64)
    N, K = W.shape
    g = W.reshape(N, K // group, group)
    fine = np.isfinite(g).all(-1)
    amax = np.where(fine, np.abs(np.where(np.isfinite(g), g, 0.0)).max(-1), 0.0)
    scale = np.maximum(round_scale(amax / 7.0), least)
    code = 8 + np.clip(np.rint(np.where(fine[..., None], g, 0.0) / scale[..., None]), -7, 7)
    return code.reshape(N, K).astype(np.int64), np.where(fine, scale, np.nan)


def w4_pack(code):
    """Two codes along K to a byte, the even k in the low half."""
    code = np.asarray(code)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def w4_weight(q, scales, zeros=None):
    """The weight [N, K] that packed codes, scales and zero points stand for."""
    q = np.asarray(q).astype(np.int64)
    code = np.empty((q.shape[0], q.shape[1] * 2))
    code[:, 0::2] = q & 15
    code[:, 1::2] = q >> 4
    scales = np.asarray(scales, dtype=np.float64)
    group = code.shape[1] // scales.shape[1]
    z = np.full(scales.shape, 8.0) if zeros is None else np.asarray(zeros, dtype=np.float64)
    return (code - np.repeat(z, group, 1)) * np.repeat(scales, group, 1)


def rope(x, positions, inv_freq, axis_of, interleaved=False, inverse=False):
    """x [rows, heads, D] with its first 2 * len(inv_freq) channels rotated; positions [axes, rows] integers."""
    x = np.asarray(x, dtype=np.float64)
    n = len(inv_freq)
    # (a 31-bit position times a 24-bit frequency: 55 bits, rounded at 2^-53 of the angle)
    t = np.empty((x.shape[0], n))
    for i in range(n):
        p = np.asarray(positions)[axis_of[i]].astype(np.float64)
        t[:, i] = p * float(inv_freq[i])
    if inverse:
        t = -t
    c, s = np.cos(t)[:, None, :], np.sin(t)[:, None, :]
    y = x.copy()
    lo = np.arange(n) * (2 if interleaved else 1)
    hi = lo + (1 if interleaved else n)
    a, b = x[..., lo], x[..., hi]
    y[..., lo] = a * c - b * s
    y[..., hi] = b * c + a * s
    return y


def e4m3_round(y):
    """Nearest value of the finite 8-bit float with 4 exponent and 3 mantissa bits, ties to even."""
    y = np.asarray(y, dtype=np.float64)
    _, e = np.frexp(np.abs(y))  # |y| = m 2^e, m in [0.5, 1)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.rint(y / step) * step, -448.0, 448.0)


def kv_quantize(x, fmt):
    """Codes (as the numbers they are) and fp32 scales of head rows x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    fine = np.isfinite(x).all(-1)
    x = np.where(fine[..., None], x, 0.0)
    inv = np.float32(1.0) / np.float32(KV_TOP[fmt])
    scale = np.maximum(np.abs(x).max(-1).astype(np.float32) * inv, np.float32(KV_TINY)).astype(np.float64)
    y = x / scale[..., None]
    code = np.clip(np.rint(y), -127, 127) if fmt == "int8" else e4m3_round(y)
    return code, np.where(fine, scale, np.nan)


def kv_places(rows, n_seqs, page_size, n_pages, page_table, cu_rows=None, start=None):
    """For each row: (page, row in the page), None if it belongs to no sequence, "bad" if its position has no page."""
    out = []
    for i in range(rows):
        if cu_rows is None:
            b, pos = (i, 0) if i < n_seqs else (None, 0)
        else:
            b = next((b for b in range(n_seqs) if cu_rows[b] <= i < cu_rows[b + 1]), None)
            pos = 0 if b is None else i - int(cu_rows[b])
        if b is None:
            out.append(None)
            continue
        pos += 0 if start is None else int(start[b])
        table = page_table[b]
        if pos < 0 or pos >= len(table) * page_size:
            out.append("bad")
            continue
        page = int(table[pos // page_size])
        out.append((page, pos % page_size) if 0 <= page < n_pages else "bad")
    return out
