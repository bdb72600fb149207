"""The block-scaled 4-bit cache in NumPy, from its definition.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A value is code * block scale * tensor scale (E2M1 codes, an E4M3 scale for 16
consecutive dims).  ``quantise`` follows the stated float32 steps with searches
among the representable values; ``pack`` / ``unpack`` place rows into the byte
tiles by an index formula per byte; attention dequantises every row (code *
scale is exact in float32) and runs the float64 C oracle on the result.
"""
from __future__ import annotations

import numpy as np

import oracle
from oracle import twin

CODE_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALE_VALUES = twin.e4m3_values()[:127]      # the finite non-negative scales, increasing


def _nearest(x, grid):
    """Index of the grid value nearest to x >= 0, ties to the even index,
    saturating (NaN gives index 0)."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    below, above = x - grid[lo], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(np.isnan(x), 0, np.where(up, hi, lo)).astype(np.uint8)


def quantise(rows: np.ndarray, tensor_scale: float):
    """float32 rows [..., D] -> (codes [..., D] uint8 0..15, scale bytes [..., D / 16])."""
    t = np.float32(tensor_scale)
    x = np.asarray(rows, dtype=np.float32).reshape(rows.shape[:-1] + (-1, 16))
    with np.errstate(all="ignore"):
        ideal = np.abs(x).max(-1) / t / np.float32(6)         # np.max keeps a NaN
        byte = np.where(np.isnan(ideal), 0x7F, _nearest(ideal, SCALE_VALUES)).astype(np.uint8)
        factor = twin.e4m3_values()[byte].astype(np.float32) * t
        y = x / factor[..., None]
        live = (factor > 0)[..., None]
        code = np.where(live, _nearest(np.abs(y), CODE_VALUES) | (np.signbit(y) << 3), 0)
    return code.astype(np.uint8).reshape(rows.shape), byte


def code_value(codes):
    v = CODE_VALUES[codes & 7]
    return np.where(codes & 8, -v, v)


def code_place(D: int, keys: bool):
    """Byte of the tile that holds the code of (row, dim): [16, D]."""
    r, d = np.arange(16)[:, None], np.arange(D)[None]
    if keys:
        P = min(D, 128)
        return (d // P) * (8 * P) + r * (P // 2) + (d % P) // 2
    return (d // 8) * 64 + r * 4 + (d % 8) // 2


def scale_place(D: int, keys: bool):
    """Byte of the tile that holds the scale of (row, block): [16, D / 16]."""
    r, k = np.arange(16)[:, None], np.arange(D // 16)[None]
    return 8 * D + (r * (D // 16) + k if keys else k * 16 + r)


def head_dim(cache: np.ndarray) -> int:
    return cache.shape[-1] * 16 // 9


def write_rows(cache: np.ndarray, slots, codes, scales, keys: bool) -> None:
    """Rows (codes [T, Hkv, D], scales [T, Hkv, D / 16]) into slots >= 0 of the
    cache [NB, Hkv, 16, 9 D / 16], in place."""
    D = head_dim(cache)
    tiles = cache.reshape(cache.shape[0], cache.shape[1], 9 * D)
    cp, sp = code_place(D, keys), scale_place(D, keys)
    for t, s in enumerate(np.asarray(slots)):
        if 0 <= s < cache.shape[0] * 16:
            blk, row = divmod(int(s), 16)
            tiles[blk][:, cp[row, ::2]] = codes[t][:, ::2] | (codes[t][:, 1::2] << 4)
            tiles[blk][:, sp[row]] = scales[t]


def append(k_cache, v_cache, k_new, v_new, slots, k_scale, v_scale) -> None:
    """The quantising append, in place; k_new / v_new float32 [T, Hkv, D]."""
    write_rows(k_cache, slots, *quantise(k_new, k_scale), True)
    write_rows(v_cache, slots, *quantise(v_new, v_scale), False)


def unpack(cache: np.ndarray, keys: bool) -> np.ndarray:
    """code * block scale of every row, float64 [NB, Hkv, 16, D]."""
    D = head_dim(cache)
    tiles = cache.reshape(cache.shape[0], cache.shape[1], 9 * D)
    byte = tiles[..., code_place(D, keys)]
    code = np.where(np.arange(D) % 2 == 1, byte >> 4, byte & 15)
    scale = twin.e4m3_values()[tiles[..., scale_place(D, keys)]]
    return code_value(code) * np.repeat(scale, 16, axis=-1)


def load(cache, slots, tensor_scale, keys: bool) -> np.ndarray:
    """Rows of the slots, float32 [T, Hkv, D]: (code * scale) * tensor scale."""
    rows = unpack(cache, keys).transpose(0, 2, 1, 3)          # [NB, 16, Hkv, D]
    slots = np.asarray(slots)
    inside = (slots >= 0) & (slots < cache.shape[0] * 16)
    s = np.where(inside, slots, 0)
    x = rows[s // 16, s % 16].astype(np.float32) * np.float32(tensor_scale)
    return np.where(inside[:, None, None], x, np.float32(0))


def attention(q, k_cache, v_cache, block_table, context_lens, scale, k_scale, v_scale,
              tree_mask=None) -> np.ndarray:
    """Float64 output [B, Q, Hq, D]; q float32 [B, Q, Hq, D] (exact widening)."""
    k = np.ascontiguousarray(unpack(k_cache, True), dtype=np.float32)
    v = np.ascontiguousarray(unpack(v_cache, False), dtype=np.float32)
    q = np.ascontiguousarray(q, dtype=np.float32)
    s = float(scale) * float(np.float32(k_scale))
    if tree_mask is None:
        o = oracle.paged_attention(q, k, v, block_table, context_lens, s, "f32")
    else:
        o = oracle.tree_attention(q, k, v, block_table, context_lens, s, "f32", tree_mask)
    return o * float(np.float32(v_scale))


def pack(rows: np.ndarray, tensor_scale: float, keys: bool) -> np.ndarray:
    """A cache [NB, Hkv, 16, 9 D / 16] holding the float32 rows [NB, Hkv, 16, D];
    rows of NaN become bytes that stand for nothing (all ones)."""
    NB, H, _, D = rows.shape
    codes, scales = quantise(rows, tensor_scale)
    none = np.isnan(rows).all(-1)
    byte = codes[..., ::2] | (codes[..., 1::2] << 4)
    byte[none], scales[none] = 255, 255
    tiles = np.zeros((NB, H, 9 * D), np.uint8)
    tiles[..., code_place(D, keys)[:, ::2]] = byte
    tiles[..., scale_place(D, keys)] = scales
    return tiles.reshape(NB, H, 16, 9 * D // 16)
