"""Oracle (float64, numpy): window attention with sinks over a paged cache, and what an fp8 or NVFP4
cache may hold for given K / V rows. Written from the definitions; shares nothing with the kernels."""
from __future__ import annotations

import numpy as np

from .formats import bf16_bits_to_float, e2m1_to_float, e4m3_to_float, nvfp4_slot_rows

BLOCK, ROWS, D = 128, 16, 128


def visible(pos: int, window: int, num_sinks: int) -> np.ndarray:
    """The keys a query at `pos` sees: n <= pos and (n > pos - window, any n for window 0, or n < num_sinks)."""
    n = np.arange(max(pos + 1, 0))
    return n if window == 0 else n[(n > pos - window) | (n < num_sinks)]


def rows_of(cache: np.ndarray, kv_dtype: str, num_kv_heads: int, pages: np.ndarray, rows: np.ndarray):
    """K and V [n, Hkv, 128] float64 of the page rows; cache uint8 [pages, bytes]."""
    k = np.empty((len(pages), num_kv_heads, D))
    v = np.empty_like(k)
    for i, (p, r) in enumerate(zip(pages, rows)):
        page = cache[p]
        for g in range(num_kv_heads):
            if kv_dtype == "nvfp4":
                k[i, g] = nvfp4_slot_rows(page[(2 * g) * 1152:(2 * g + 1) * 1152], np.array([r]))[0]
                v[i, g] = nvfp4_slot_rows(page[(2 * g + 1) * 1152:(2 * g + 2) * 1152], np.array([r]))[0]
                continue
            width = 4 * D if kv_dtype == "bf16" else 2 * D
            raw = page[(g * ROWS + r) * width:(g * ROWS + r + 1) * width]
            row = bf16_bits_to_float(raw.view(np.uint16)) if kv_dtype == "bf16" else e4m3_to_float(raw)
            k[i, g], v[i, g] = row[:D], row[D:]
    return k, v


def window_row(q, cache, kv_dtype, num_kv_heads, table_row, pos, window, num_sinks, scale, k_scale, v_scale,
               block_page_stride=8):
    """One query row q [Hq, 128]: (out [Hq, 128], lse [Hq], mass [Hq, 128], zabs [Hq]).

    mass = v_scale * sum p |v| and zabs = the largest scale * sum_d |q_d k_d| of a visible key bound
    what rounding p and the logits can move the result by."""
    hq = q.shape[0]
    keys = visible(pos, window, num_sinks)
    if len(keys) == 0:
        return np.zeros((hq, D)), np.full(hq, -np.inf), np.zeros((hq, D)), np.zeros(hq)
    pages = np.asarray(table_row)[keys // BLOCK].astype(np.int64) * block_page_stride + keys % BLOCK // ROWS
    k, v = rows_of(cache, kv_dtype, num_kv_heads, pages, keys % ROWS)
    g = hq // num_kv_heads
    k, v = np.repeat(k, g, 1), np.repeat(v, g, 1)
    z = np.einsum("hd,nhd->hn", q, k) * (scale * k_scale)
    zabs = np.einsum("hd,nhd->hn", np.abs(q), np.abs(k)).max(1) * abs(scale * k_scale)
    top = z.max(1, keepdims=True)
    e = np.exp(z - top)
    s = e.sum(1, keepdims=True)
    p = e / s
    return (v_scale * np.einsum("hn,nhd->hd", p, v), (top + np.log(s))[:, 0],
            abs(v_scale) * np.einsum("hn,nhd->hd", p, np.abs(v)), zabs)


def e4m3_values():
    """The 127 finite non-negative e4m3 values, ascending (index = code)."""
    return e4m3_to_float(np.arange(127))


def e2m1_values():
    """The 8 non-negative e2m1 values, ascending (index = code)."""
    return e2m1_to_float(np.arange(8))


def nearest(x, values):
    """Index of the value nearest to x >= 0, ties to the even index, saturating."""
    i = np.clip(np.searchsorted(values, x, side="right") - 1, 0, len(values) - 2)
    below, above = x - values[i], values[i + 1] - x
    return i + ((below > above) | ((below == above) & (i % 2 == 1)))
