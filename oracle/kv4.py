"""The paged 4-bit cache in plain NumPy: quantization, layout, rotation, attention (float64).

A vector x is held as m + s c: m = min(x) rounded down to bf16, s = (max(x) - m) / 15 rounded up to
bf16 (float32 difference and quotient, at least the smallest normal float32, 0 when max(x) = m),
c = (x - m) / s rounded to nearest, ties to even. A vector with a value that is not finite, or whose
range max(x) - m is no finite float32, is held as NaN (m) with s = 0 and codes 0.

A block of 16 tokens of one head: 16 rows of key codes (d / 2 bytes), 16 of value codes, 16 key pairs,
16 value pairs; coordinate 2j in the low half of byte j; the 16-byte chunk at place p of row t is chunk
p ^ x(t), x(t) = (t d / 256) mod (d / 32); a pair is s | m << 16 as bf16 bits, little-endian.
Pages: [n_pages][heads][page_tokens / 16][16 d + 128].
"""

from __future__ import annotations

import math

import numpy as np

TINY = float(np.finfo(np.float32).tiny)


def bf16_bits(x, up: bool) -> np.ndarray:
    """bf16 bit pattern of float32 values, rounded toward +inf (up) or -inf, through float64 arithmetic."""
    x = np.asarray(x, np.float32)
    bits = x.view(np.uint32).astype(np.int64)
    cand = [((bits >> 16) + k) << 16 for k in (0, 1)]          # the two neighbours in magnitude
    vals = [np.asarray(c, np.uint32).view(np.float32).astype(np.float64) for c in cand]
    exact = x.astype(np.float64)
    toward_zero_ok = (vals[0] >= exact) if up else (vals[0] <= exact)
    return np.where(toward_zero_ok, cand[0] >> 16, cand[1] >> 16).astype(np.uint32)


def bf16_value(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint32) << np.uint32(16)).view(np.float32)


def quantize(x) -> tuple[np.ndarray, np.ndarray, np.ndarray]:
    """(codes uint8 [..., d], s bits, m bits [...]) of float32 vectors x [..., d]."""
    x = np.asarray(x, np.float32)
    finite = np.isfinite(x).all(-1)
    z = np.where(finite[..., None], x, np.float32(0))
    mb = bf16_bits(z.min(-1), up=False)
    m = bf16_value(mb)
    with np.errstate(over="ignore", invalid="ignore"):
        r = z.max(-1) - m
        q = np.maximum(r / np.float32(15), np.float32(TINY))
    ok = finite & np.isfinite(r)
    live = ok & (r > 0)
    sb = np.where(live, bf16_bits(np.where(live, q, np.float32(1)), up=True), 0).astype(np.uint32)
    s = bf16_value(sb)
    with np.errstate(over="ignore", invalid="ignore"):
        e = (z - m[..., None]).astype(np.float32).astype(np.float64)
        c = np.rint(e / np.where(live, s, 1.0).astype(np.float64)[..., None])
    codes = np.where(live[..., None], np.clip(c, 0, 15), 0).astype(np.uint8)
    return codes, sb, np.where(ok, mb, 0x7FC0).astype(np.uint32)


def values(codes, sb, mb) -> np.ndarray:
    """float64 m + s c."""
    return bf16_value(mb).astype(np.float64)[..., None] + bf16_value(sb).astype(np.float64)[..., None] * codes


def block_bytes(d: int) -> int:
    return 16 * d + 128


def _row_bytes(codes_row: np.ndarray, t: int, d: int) -> np.ndarray:
    raw = codes_row[0::2] | (codes_row[1::2] << 4)
    chunks = raw.reshape(d // 32, 16)
    x = (t * d // 256) % (d // 32)
    return np.concatenate([chunks[p ^ x] for p in range(d // 32)])


def store(pages: np.ndarray, page: int, head: int, slot: int, side: int, codes, sb, mb) -> None:
    """Writes one vector into a pool uint8 [n_pages, heads, page_tokens / 16, 16 d + 128]; side 0 key, 1 value."""
    d = len(codes)
    blk, t = pages[page, head, slot // 16], slot % 16
    at = side * 8 * d + t * (d // 2)
    blk[at:at + d // 2] = _row_bytes(np.asarray(codes, np.uint8), t, d)
    at = 16 * d + side * 64 + 4 * t
    word = int(sb) | (int(mb) << 16)
    blk[at:at + 4] = np.frombuffer(np.array([word], "<u4").tobytes(), np.uint8)


def load(pages: np.ndarray, page: int, head: int, slot: int, side: int):
    """(codes, s bits, m bits) of one vector of the pool."""
    d = (pages.shape[-1] - 128) // 16
    blk, t = pages[page, head, slot // 16], slot % 16
    x = (t * d // 256) % (d // 32)
    chunks = blk[side * 8 * d + t * (d // 2):][:d // 2].reshape(d // 32, 16)
    raw = np.concatenate([chunks[p ^ x] for p in range(d // 32)])
    codes = np.empty(d, np.uint8)
    codes[0::2], codes[1::2] = raw & 15, raw >> 4
    word = int(np.frombuffer(blk[16 * d + side * 64 + 4 * t:][:4].tobytes(), "<u4")[0])
    return codes, word & 0xFFFF, word >> 16


def rope_table(n_pos: int, rot: int, theta: float = 10000.0) -> np.ndarray:
    ang = np.arange(n_pos)[:, None] * theta ** (-np.arange(0, rot, 2) / rot)[None, :]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def rotate(x, table, pos: int, interleaved: bool, round_to) -> np.ndarray:
    """float32 heads x [heads, d] turned by position pos, every operation rounded to float32, then round_to."""
    x = np.asarray(x, np.float32)
    if table is None:
        return x
    h = table.shape[1] // 2
    c, s = table[pos, :h], table[pos, h:]
    y = x.copy()
    a, b = (x[:, 0:2 * h:2], x[:, 1:2 * h:2]) if interleaved else (x[:, :h], x[:, h:2 * h])
    ya, yb = a * c - b * s, b * c + a * s
    if interleaved:
        y[:, 0:2 * h:2], y[:, 1:2 * h:2] = ya, yb
    else:
        y[:, :h], y[:, h:2 * h] = ya, yb
    y[:, :2 * h] = round_to(y[:, :2 * h])
    return y


def attend(q, keys, vals, scale: float, spread=None):
    """(output [d], log-sum-exp, sum of p |spread|) of one float64 query over keys [n, d] and values [n, d]."""
    if len(keys) == 0:
        return np.zeros(vals.shape[-1]), -math.inf, np.zeros(vals.shape[-1])
    s = scale * (keys @ q)
    top = s.max()
    p = np.exp(s - top)
    total = p.sum()
    p = p / total
    return p @ vals, top + math.log(total), (p @ spread if spread is not None else None)
