"""Plain 64-bit references of the quantised cache and of attention with
modified scores, written from their formulas (no code of the library)."""
from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TINY = np.float32(2.0 ** -80)


def e4m3_values() -> np.ndarray:
    """The value of every e4m3 code, in 64 bits."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        x = np.nan if c & 127 == 127 else x
        v[c] = -x if c >= 128 else x
    return v


def nearest_even(x: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the table's (ascending) value nearest to x >= 0, ties to the
    even index, values past the last to the last."""
    i = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo, hi = table[i - 1], table[i]
    down = (x - lo < hi - x) | ((x - lo == hi - x) & ((i - 1) % 2 == 0))
    return np.where(down, i - 1, i)


def quantise_row(x: np.ndarray, fmt: str):
    """(codes, group scale codes, row scale) of one binary32 row, the products
    and divisions in binary32 as the format says."""
    x = x.astype(np.float32)
    D = x.size
    if not np.isfinite(x).all():
        nan = np.uint32(0x7FC00000).view(np.float32)
        return (np.full(D, 128, np.uint8) if fmt == "int8" else np.zeros(D, np.uint8)), np.zeros(D // 16, np.uint8), nan
    a = np.abs(x).max()
    if a < TINY:
        return (np.full(D, 128, np.uint8) if fmt == "int8" else np.zeros(D, np.uint8)), np.zeros(D // 16, np.uint8), np.float32(0)
    if fmt == "int8":
        s = np.float32(a * np.float32(1 / 127))
        return (np.rint(x / s).astype(np.int32) + 128).astype(np.uint8), None, s
    s = np.float32(a * np.float32(1 / 2688))
    table = e4m3_values()[:127]
    codes, groups = np.zeros(D, np.uint8), np.zeros(D // 16, np.uint8)
    for j in range(D // 16):
        g = x[16 * j: 16 * j + 16]
        t = int(nearest_even(np.float64(np.abs(g).max() / np.float32(np.float32(6) * s)), table))
        groups[j] = t
        step = np.float32(np.float32(table[t]) * s)
        if step > 0:
            y = (g / step).astype(np.float32)
            codes[16 * j: 16 * j + 16] = nearest_even(np.abs(y).astype(np.float64), E2M1) | (np.signbit(y) << 3)
    return codes, groups, s


def row_bytes(d: int, fmt: str) -> int:
    return d if fmt == "int8" else d // 2


def write_row(tile: np.ndarray, off: int, x: np.ndarray, bs: int, fmt: str) -> None:
    """Quantise the row into position `off` of a tile's bytes."""
    d, row = x.size, row_bytes(x.size, fmt)
    codes, groups, s = quantise_row(x, fmt)
    packed = codes if fmt == "int8" else codes[0::2] | (codes[1::2] << 4)
    for c in range(row // 16):
        at = off * row + 16 * (c ^ ((off * row // 128) % (row // 16)))
        tile[at: at + 16] = packed[16 * c: 16 * c + 16]
    if fmt == "fp4":
        at = bs * row + off * (d // 16)
        tile[at: at + d // 16] = groups
    at = tile.size - 4 * bs + 4 * off
    tile[at: at + 4] = np.array([s], np.float32).view(np.uint8)


def read_row(tile: np.ndarray, off: int, d: int, bs: int, fmt: str) -> np.ndarray:
    """The row's values in 64 bits."""
    row = row_bytes(d, fmt)
    packed = np.concatenate([tile[off * row + 16 * p: off * row + 16 * p + 16]
                             for p in ((c ^ ((off * row // 128) % (row // 16))) for c in range(row // 16))])
    at = tile.size - 4 * bs + 4 * off
    s = np.float64(tile[at: at + 4].copy().view(np.float32)[0])
    if fmt == "int8":
        return (packed.astype(np.float64) - 128) * s
    nib = np.stack([packed & 15, packed >> 4], 1).reshape(-1)
    v = np.where(nib >= 8, -E2M1[nib & 7], E2M1[nib & 7])
    t = e4m3_values()[tile[bs * row + off * (d // 16): bs * row + (off + 1) * (d // 16)]]
    return v * np.repeat(t, 16) * s


def attention_row(q, K, V, p, L, scale, cap=0.0, slope=0.0, window=0, sinks=0, prefix=0, missing=()):
    """One query row at position p over K, V [L, D] (64 bits); `missing`
    positions are left out."""
    t = np.arange(L)
    keep = t <= p
    if window:
        keep &= (t > p - window) | (t < sinks)
    keep |= t < prefix
    if len(missing):
        keep[list(missing)] = False
    if not keep.any():
        return np.zeros(V.shape[1])
    x = scale * (K[keep] @ q)
    if cap:
        x = cap * np.tanh(x / cap)
    x = x - slope * np.abs(p - t[keep])
    w = np.exp(x - x.max())
    return (w / w.sum()) @ V[keep]


def tables_for(lens, bs, gen, spare=3):
    """A shuffled pool's block tables for the lengths, unused entries outside
    the pool; (int32 tables, blocks in the pool)."""
    nb = [-(-n // bs) for n in lens]
    pool = sum(nb) + spare
    ids = torch.randperm(pool, generator=gen)
    tables = torch.full((len(lens), max(1, max(nb, default=1)) + 1), 0x7FFFFFFF, dtype=torch.int32)
    at = 0
    for i, n in enumerate(nb):
        tables[i, :n] = ids[at: at + n].to(torch.int32)
        at += n
    return tables, pool


def slots_for(lens, tables, bs):
    s = [int(tables[i, p // bs]) * bs + p % bs for i, n in enumerate(lens) for p in range(n)]
    return torch.tensor(s, dtype=torch.int64)
