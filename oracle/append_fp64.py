"""CPU oracle of the append calls: rotary embedding, page scales and the store
into a paged cache, in fp64.

TEST INFRASTRUCTURE ONLY (see attention_fp64.py): NumPy, shares no code with
the CUDA path.

Token t of sequence b (L new of S cached tokens) is stored at position
S - L + t. A pair of a head's columns turns as the complex number
(x1 + i x2) e^{i angle}. A page-scaled cache holds code * scale: the scale of
a (page, head) that gets new tokens is the smallest 2^e, -64 <= e <= 64, with
max|new| <= 448 * 2^e, or the page's earlier scale if older tokens precede
the new ones and theirs is larger.
"""
from __future__ import annotations

import math

import numpy as np

PAGE_SIZE = 16
MIN_SCALE, MAX_SCALE = 2.0 ** -64, 2.0 ** 64


def page_scale(amax: float) -> float:
    """The smallest 2^e, -64 <= e <= 64, with amax <= 448 * 2^e."""
    e = -64
    while e < 64 and amax > math.ldexp(448.0, e):
        e += 1
    return math.ldexp(1.0, e)


def usable(scale: float) -> float:
    """A stored page scale as it is read: clamped, NaN as the smallest."""
    return MIN_SCALE if math.isnan(scale) else min(max(scale, MIN_SCALE), MAX_SCALE)


def rotated(x: np.ndarray, cos_sin: np.ndarray, position: int, interleaved: bool) -> np.ndarray:
    """Rows x [..., dim] turned by the angles of one position (clamped into the table)."""
    y = np.array(x, dtype=np.float64)
    if cos_sin is None:
        return y
    rot = cos_sin.shape[1]
    half = rot // 2
    row = np.asarray(cos_sin, dtype=np.float64)[min(max(position, 0), cos_sin.shape[0] - 1)]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        x1, x2 = y[..., a].copy(), y[..., b].copy()
        y[..., a] = x1 * row[i] - x2 * row[half + i]
        y[..., b] = x2 * row[i] + x1 * row[half + i]
    return y


class Store:
    """What a cache holds after the call: ``value`` (the fp64 number a slot
    stands for, saturated as the type does; NaN where nothing was written) and
    ``written``; for a page-scaled cache ``scales`` after the call and ``kept``
    (older tokens, held under a scale that may have grown)."""

    def __init__(self, pages, heads, dim, scales=None):
        self.value = np.full((pages, PAGE_SIZE, heads, dim), np.nan)
        self.written = np.zeros((pages, PAGE_SIZE), dtype=bool)
        self.kept = np.zeros((pages, PAGE_SIZE), dtype=bool)
        self.scales = None if scales is None else np.array(scales, dtype=np.float64)


def append_oracle(rows, block_table, cu_seqlens_q, seqused_k, num_pages, before=None, scales=None,
                  descale=None, limit=math.inf):
    """Stores rows [T, heads, dim] (already rotated, fp64). ``before``: the
    codes' values [pages, 16, heads, dim] before the call (page-scaled caches);
    ``limit``: the largest stored code (448 for e4m3)."""
    rows = np.asarray(rows, dtype=np.float64)
    heads, dim = rows.shape[1:]
    st = Store(num_pages, heads, dim, scales)
    with np.errstate(invalid="ignore", over="ignore"):
        for b in range(len(seqused_k)):
            a, z = int(cu_seqlens_q[b]), int(cu_seqlens_q[b + 1])
            L, S = z - a, int(seqused_k[b])
            byp = {}
            for t in range(L):
                x = S - L + t
                if x < 0 or x // PAGE_SIZE >= block_table.shape[1]:
                    continue
                page = int(block_table[b, x // PAGE_SIZE])
                if 0 <= page < num_pages:
                    byp.setdefault(page, []).append((x % PAGE_SIZE, a + t))
            for page, toks in byp.items():
                first = min(s for s, _ in toks)
                for h in range(heads):
                    if scales is None:
                        s = 1.0 if descale is None else float(descale)
                    else:
                        fin = np.abs(np.concatenate([rows[r, h] for _, r in toks]))
                        s = page_scale(float(np.nanmax(fin)) if not np.isnan(fin).all() else 0.0)
                        if first > 0:
                            had = usable(float(scales[page, h]))
                            s = max(s, had)
                            st.value[page, :first, h] = before[page, :first, h] * had
                            st.kept[page, :first] = True
                        st.scales[page, h] = s
                    for slot, r in toks:
                        code = rows[r, h] / s
                        st.value[page, slot, h] = np.where(np.isnan(code), np.nan, np.clip(code, -limit, limit)) * s
                        st.written[page, slot] = True
    return st
