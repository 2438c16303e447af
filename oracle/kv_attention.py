"""Plain statement of the paged key/value cache and its attention (numpy).

Stored values follow include/rg.h's rg_kv_write, the bytes of a page the
layout that csrc/rg_kv.cuh describes, each byte placed by its own index;
the attention is the definition's sum in 64 bits.
"""
from __future__ import annotations

import numpy as np

from .quant_out_prod import BF16, F16, Q4_0, Q8_0

GRANULE = 16


def kv_row_bytes(wtype: int, D: int) -> int:
    return {F16: 2 * D, BF16: 2 * D, Q8_0: D // 32 * 34, Q4_0: D // 32 * 18}[wtype]


def kv_page_bytes(wtype: int, D: int, H: int, P: int) -> int:
    return 2 * H * P * kv_row_bytes(wtype, D)


def bf16_round(x: np.ndarray) -> np.ndarray:
    """F32 -> bfloat16 bits, to nearest even (NaN stays NaN)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((u >> 16) + ((u & 0xFFFF) + ((u >> 16) & 1) > 0x8000)).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FFF), r)


def kv_quantise(wtype: int, x: np.ndarray):
    """Rows [..., D] F32 -> (codes [..., D] uint8, scales [..., D/32] fp16)."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 32)
    mag = np.abs(b)
    big = mag.max(-1, keepdims=True)          # NaN if there is one
    fine = np.isfinite(b).all(-1, keepdims=True)
    with np.errstate(all="ignore"):
        if wtype == Q8_0:
            top, steps = big, np.float32(127)
        else:
            first = np.argmax(mag == big, -1)[..., None]
            top, steps = np.take_along_axis(b, first, -1), np.float32(-8)
        d = (top / steps).astype(np.float16)
        inv = np.where(fine & (d != 0), steps / top, np.float32(0)).astype(np.float32)
        r = np.where(inv == 0, np.float32(0), np.rint(b * inv))
    d = np.where(fine, d, np.array(0x7E00, np.uint16).view(np.float16))
    if wtype == Q8_0:
        codes = r.astype(np.int32).astype(np.int8).view(np.uint8)
    else:
        codes = np.clip(r + 8, 0, 15).astype(np.uint8)
    return codes.reshape(x.shape), d[..., 0]


def kv_values(wtype: int, x: np.ndarray) -> np.ndarray:
    """What rows [..., D] F32 stand for once stored, F32 (exact)."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        if wtype == F16:
            return x.astype(np.float16).astype(np.float32)
        if wtype == BF16:
            return (bf16_round(x).astype(np.uint32) << 16).view(np.float32)
        codes, d = kv_quantise(wtype, x)
        q = codes.view(np.int8).astype(np.float32) if wtype == Q8_0 else codes.astype(np.float32) - 8
        return q * np.repeat(d.astype(np.float32), 32, -1)


def kv_places(wtype: int, D: int, kind: int, j: int):
    """(byte offset of each dimension's code, which half of the byte, byte offset
    of each block's scale) of token j of a granule."""
    d = np.arange(D)
    c, e, q, g, t = d // 32, d % 8, d // 8 % 4, d % 8, d // 8 % 4
    a, n, b, k = j // 4, j // 2 % 2, j % 2, j % 4
    half = np.zeros(D, int)
    if wtype in (F16, BF16):
        if kind == 0:
            at = (((c * 2 + n) * 8 + 2 * a + b) * 4 + t) * 16 + 2 * e
        else:
            at = ((d // 16 * 8 + g) * 4 + a) * 16 + q % 2 * 8 + 2 * k
        return at, half, None
    lane = (2 * a + b) * 4 + t if kind == 0 else g * 4 + a
    if wtype == Q8_0:
        at = c * 512 + lane * 16 + (n * 8 + e if kind == 0 else q * 4 + k)
    elif kind == 0:
        nibble = e % 2 * 4 + e // 2
        at, half = c * 256 + lane * 8 + n * 4 + nibble // 2, nibble % 2
    else:
        nibble = k % 2 * 4 + k // 2 * 2 + q % 2
        at, half = c * 256 + lane * 8 + q // 2 * 4 + nibble // 2, nibble % 2
    blk = np.arange(D // 32)
    codes = 16 * D if wtype == Q8_0 else 8 * D
    return at, half, codes + 2 * (16 * blk + (2 * (2 * a + b) + n if kind == 0 else j))


def kv_store(pool: np.ndarray, wtype: int, D: int, H: int, P: int, page: int, pos: int, kind: int, head: int,
             x: np.ndarray) -> None:
    """One token's row x [D] F32 into pool [pages, page bytes] uint8."""
    rb = kv_row_bytes(wtype, D)
    base = (kind * H + head) * P * rb + pos % P // GRANULE * GRANULE * rb
    at, half, scale = kv_places(wtype, D, kind, pos % GRANULE)
    row = pool[page]
    if wtype in (F16, BF16):
        bits = np.asarray(x, np.float32).astype(np.float16).view(np.uint16) if wtype == F16 else bf16_round(x)
        row[base + at], row[base + at + 1] = bits & 255, bits >> 8
        return
    codes, d = kv_quantise(wtype, x)
    if wtype == Q8_0:
        row[base + at] = codes
    else:
        for h in (0, 1):
            w = at[half == h]
            row[base + w] = (row[base + w] & (0xF0 if h == 0 else 0x0F)) | (codes[half == h] << (4 * h))
    bits = d.view(np.uint16)
    row[base + scale], row[base + scale + 1] = bits & 255, bits >> 8


def kv_attend(q, K, V, pos, scale, window=0):
    """out [n, Hq, D] and its absolute sum sum_j w_j |v_j| / sum_j w_j, of rows at
    positions pos [n] over K, V [L, H, D] (64 bits); rows that see nothing: 0.
    Values at hidden positions do not enter, whatever they are."""
    q, K, V = (np.asarray(x, np.float64) for x in (q, K, V))
    n, Hq, D = q.shape
    G = Hq // K.shape[1]
    out, mag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    for i in range(n):
        lo = max(0, pos[i] - window + 1) if window else 0
        hi = min(pos[i] + 1, K.shape[0])
        if hi <= lo:
            continue
        for h in range(Hq):
            z = K[lo:hi, h // G] @ q[i, h] * scale
            with np.errstate(all="ignore"):
                w = np.exp(z - z.max())
                out[i, h] = w @ V[lo:hi, h // G] / w.sum()
                mag[i, h] = w @ np.abs(V[lo:hi, h // G]) / w.sum()
    return out, mag
