"""Float64 oracle of the 4-bit KV cache: the number format, the tile layout and attention over it.

Written from the definitions in include/pqhsa.h (4-bit KV cache), with tables and searches instead of
arithmetic on bits; test infrastructure only.
"""
from __future__ import annotations

import math

import numpy as np

TILE_TOKENS, TILE_BYTES, D, BLOCK = 16, 2304, 128, 16
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# value of every scale byte: 5 exponent bits, 3 mantissa bits, bias 15; the top exponent is infinity and NaN
SCALES = np.array([math.ldexp(b % 8, -17) if b < 8 else math.ldexp(8 + b % 8, b // 8 - 18) for b in range(248)]
                  + [math.inf] + 7 * [math.nan])
MAX_SCALE_BYTE = 226   # 10240


def _nearest(table: np.ndarray, y: np.ndarray) -> np.ndarray:
    """Index of the nearest entry of an ascending table, a tie going to the even index."""
    hi = np.clip(np.searchsorted(table, y), 1, len(table) - 1)
    lo = hi - 1
    below, above = y - table[lo], table[hi] - y
    return np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)


def quantise(x: np.ndarray):
    """Codes uint8 [..., 128] and scale bytes uint8 [..., 8] of rows of 128 (any float type)."""
    x = np.asarray(x, dtype=np.float64)
    blocks = x.reshape(x.shape[:-1] + (D // BLOCK, BLOCK))
    top = np.abs(blocks).max(-1)
    bad = ~np.isfinite(top)
    safe = np.where(bad[..., None], 0.0, blocks)
    top = np.where(bad, 0.0, top)
    # compared after multiplying by 6: every border is exact
    byte = _nearest(6 * SCALES[:MAX_SCALE_BYTE + 1], top)
    s = SCALES[byte]
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s[..., None] > 0, np.abs(safe) / s[..., None], 0.0)
    code = _nearest(MAGNITUDES, np.minimum(y, 6.0)) + 8 * np.signbit(safe)
    code = np.where(s[..., None] > 0, code, 0)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, byte).astype(np.uint8)


def values(code: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """Float64 values of codes [..., 128] and scale bytes [..., 8]."""
    v = MAGNITUDES[code & 7] * np.where(code >= 8, -1.0, 1.0)
    return (v.reshape(v.shape[:-1] + (D // BLOCK, BLOCK)) * SCALES[byte][..., None]).reshape(v.shape)


def _address(t: int, d: np.ndarray, value: bool):
    """Within a tile, of token t: byte and nibble shift of the code of dim d, and byte of its scale."""
    if not value:
        return t * 64 + d // 2, 4 * (d % 2), 2048 + 8 * (4 * (t % 8) + d // 32) + 2 * (t // 8) + d // 16 % 2
    pair = (t % 8) // 2
    return (1024 + 512 * (t // 8) + 64 * (d // 16) + 16 * pair + d % 16, np.full_like(d, 4 * (t % 2)),
            2048 + 8 * (4 * (d // 16) + pair) + 4 + 2 * (t // 8) + t % 2)


def tile_of(cache: np.ndarray, table: np.ndarray, h: int, pos: int, page_size: int) -> np.ndarray:
    """View of the tile that holds position pos of head h; cache [pages, Hkv, page_size / 16, 2304]."""
    return cache[table[pos // page_size], h, pos % page_size // TILE_TOKENS]


def put(cache, table, h, pos, page_size, k_row, v_row) -> None:
    """Write one token's key and value rows into the tile that holds it."""
    tile = tile_of(cache, table, h, pos, page_size)
    d = np.arange(D)
    for value, row in ((False, k_row), (True, v_row)):
        code, byte = quantise(row)
        at, shift, sat = _address(pos % TILE_TOKENS, d, value)
        low, high = shift == 0, shift == 4
        tile[at[low]] = (tile[at[low]] & 0xF0) | code[low]
        tile[at[high]] = (tile[at[high]] & 0x0F) | (code[high] << 4)
        tile[sat] = np.repeat(byte, BLOCK)


def get(cache, table, h, positions, page_size):
    """Float64 keys and values [n, 128] of positions of head h."""
    out = np.zeros((2, len(positions), D))
    d = np.arange(D)
    for i, pos in enumerate(positions):
        tile = tile_of(cache, table, h, int(pos), page_size)
        for value in (False, True):
            at, shift, sat = _address(int(pos) % TILE_TOKENS, d, value)
            out[int(value), i] = values((tile[at] >> shift) & 15, tile[sat[::BLOCK]])
    return out[0], out[1]


def attend(q, k, v, scale, seen):
    """Rows [n, 128] against keys and values [T, 128] under the mask seen [n, T], in float64: outputs, log of
    the sum of e^logit; a row that sees nothing gets zeros and -inf. Tokens that a row does not see do not
    enter it, whatever they hold."""
    out = np.zeros((len(q), D))
    lse = np.full(len(q), -np.inf)
    for i in range(len(q)):
        j = np.flatnonzero(seen[i])
        if len(j) == 0:
            continue
        x = scale * (k[j] @ np.asarray(q[i], dtype=np.float64))
        m = x.max()
        p = np.exp(x - m)
        out[i] = p @ v[j] / p.sum()
        lse[i] = m + np.log(p.sum())
    return out, lse
