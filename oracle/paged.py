"""Plain float64 oracle of the paged-cache operators.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The operators extend region 2 and the cache append of region 1 of the page
"DeepSpeed Inference 内核优化深度解析：多 GPU 自适应并行、算子融合推理内核与 MoQ 量化支持",
§3.2, to a cache in pages, rotary positions, grouped query heads, packed
sequences and rows of 4 bits.  The page gives no formula for any of these; the
definitions are those of include/ds_layer.h, computed here one row at a time.

Arrays are numpy float64 unless said otherwise.  Packed arrays are [tokens,
heads, d]; pages are [num_pages, kv_heads, page_size, d] (4-bit: codes uint8
[..., d / 2] with scales float16 [..., 2]).
"""
from __future__ import annotations

import numpy as np


def rotate(x, cos_sin_row, interleaved=False):
    """Rotates the first r channels of x [..., d] by the angles whose cosines
    and sines are the two halves of cos_sin_row [r]."""
    x = np.array(x, dtype=np.float64)
    cs = np.asarray(cos_sin_row, dtype=np.float64)
    half = cs.shape[0] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        x1, x2 = x[..., a].copy(), x[..., b].copy()
        x[..., a] = x1 * cs[i] - x2 * cs[half + i]
        x[..., b] = x2 * cs[i] + x1 * cs[half + i]
    return x


def quantize_u4(x):
    """Codes uint8 [..., d] (one code an element) and scales float16 [..., 2]
    (scale, minimum) of rows x [..., d], the decisions in float32."""
    x = np.asarray(x, dtype=np.float32)
    m = x.min(-1).astype(np.float16)
    m32 = m.astype(np.float32)[..., None]
    s = ((x.max(-1, keepdims=True) - m32) / np.float32(15)).astype(np.float16)
    s32 = s.astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s32 > 0, np.clip(np.rint((x - m32) / np.where(s32 > 0, s32, np.float32(1))), 0, 15), 0)
    return c.astype(np.uint8), np.concatenate([s, m[..., None]], -1)


def pack_u4(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack_u4(packed):
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def dequantize_u4(packed, scales):
    sc = np.asarray(scales, dtype=np.float64)
    return unpack_u4(packed).astype(np.float64) * sc[..., :1] + sc[..., 1:]


def place(table, page_size, b, pos):
    """(page, row in the page) of position pos of sequence b."""
    return int(table[b][pos // page_size]), pos % page_size


def positions(cu, start):
    """(row, sequence, position) of every packed row that belongs to a sequence."""
    for b in range(len(cu) - 1):
        for t in range(int(cu[b]), int(cu[b + 1])):
            yield t, b, int(start[b]) + t - int(cu[b])


def softmax_rows(s):
    """Softmax over the last axis; rows that are -inf throughout become zeros."""
    top = s.max(-1, keepdims=True)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    z = e.sum(-1, keepdims=True)
    return e / np.where(z > 0, z, 1.0)


def attend(q, k, v, first_seen, scale):
    """Causal attention of one sequence: q [Lq, heads, d] over k, v [Lk,
    kv_heads, d]; query i sees keys j < first_seen + i.  Returns out, and the
    same sum over |v| (what a relative error of the weights can move)."""
    Lq, heads, d = q.shape
    Lk, kv = k.shape[:2]
    out, mag = np.zeros((Lq, heads, d)), np.zeros((Lq, heads, d))
    seen = np.arange(Lk)[None, :] < first_seen + np.arange(Lq)[:, None]
    for h in range(heads):
        if Lk == 0:
            continue
        g = h // (heads // kv)
        p = softmax_rows(np.where(seen, scale * (q[:, h] @ k[:, g].T), -np.inf))
        out[:, h], mag[:, h] = p @ v[:, g], p @ np.abs(v[:, g])
    return out, mag


def prompt_attention(q, k, v, cu_q, cu_k, scale):
    """Packed prompts: (out, sum over |v|) [tokens, heads, d]; rows behind the
    last sequence are NaN."""
    out, mag = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for b in range(len(cu_q) - 1):
        sq, sk = slice(int(cu_q[b]), int(cu_q[b + 1])), slice(int(cu_k[b]), int(cu_k[b + 1]))
        lq, lk = sq.stop - sq.start, sk.stop - sk.start
        out[sq], mag[sq] = attend(q[sq], k[sk], v[sk], lk - lq + 1, scale)
    return out, mag


def sequence_rows(pages, table, page_size, b, n):
    """Rows 0 .. n-1 of sequence b from float64 pages: [n, kv_heads, d]."""
    rows = [pages[pg, :, r] for pg, r in (place(table, page_size, b, p) for p in range(n))]
    return np.stack(rows) if rows else np.zeros((0, pages.shape[1], pages.shape[3]))


def paged_attention(q, k_pages, v_pages, table, page_size, past, new_tokens, scale):
    """(out, sum over |v|) of `new_tokens` queries per sequence over float64 pages."""
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(len(past)):
        n = max(0, int(past[b]) + new_tokens)
        k, v = (sequence_rows(x, table, page_size, b, n) for x in (k_pages, v_pages))
        r = slice(b * new_tokens, (b + 1) * new_tokens)
        out[r], mag[r] = attend(q[r], k, v, int(past[b]) + 1, scale)
    return out, mag
