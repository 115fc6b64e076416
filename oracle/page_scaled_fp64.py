"""CPU oracle of verify attention over page-scaled e4m3 caches, in fp64, with a
bound on the kernels' own rounding.

TEST INFRASTRUCTURE ONLY (see attention_fp64.py): NumPy, shares no code with
the CUDA path.

A stored code stands for code * scale[page, head]; a scale is read as clamped
to [2^-64, 2^64], NaN as 2^-64. Attention itself is softmax_attend's.
"""
from __future__ import annotations

import numpy as np

from .attention_fp64 import PAGE_SIZE, first_visible_key, softcapped, visible_keys

MIN_SCALE, MAX_SCALE = 2.0 ** -64, 2.0 ** 64
BLOCK = 32  # keys that share a block scale of P


def read_scales(scales: np.ndarray) -> np.ndarray:
    s = np.asarray(scales, dtype=np.float64)
    return np.where(np.isnan(s), MIN_SCALE, np.clip(s, MIN_SCALE, MAX_SCALE))


def page_scaled_oracle(q, k, v, k_scales, v_scales, block_table, cu_seqlens_q, seqused_k, scale,
                       window_left=-1, softcap=0.0, sinks=None):
    """q [T, Hq, Dk], k [pages, 16, Hkv, Dk], v [pages, 16, Hkv, Dv] (code
    values, fp64), scales [pages, Hkv]. Returns (out, tol), [T, Hq, Dv] each.

    tol bounds what the kernels' roundings may add, element by element:
    * Q is two e4m3 terms, within 2^-8 of each column, so a logit moves by at
      most d = 2^-8 |scale| sum|q_c k_c| (and by tanh.approx's 2^-11 of the
      logit with a soft cap), a weight by e^{2 d} - 1 of itself;
    * P is two e4m3 terms, within 2^-8 of a weight, and rounded in steps that are
      at most 2^-21 of the largest weight times value scale among the 32 keys
      (counted from the sequence's start) that share a block scale: half a step
      a key. Blocks under 2^-115 of the row's largest fade out;
    * fp32 accumulation over n keys, n 2^-24, and the output's half step 2^-8."""
    T, Hq = q.shape[:2]
    Hkv = k.shape[2]
    G = Hq // Hkv
    out = np.zeros((T, Hq, v.shape[3]))
    tol = np.zeros_like(out)
    for b in range(len(seqused_k)):
        a, z = int(cu_seqlens_q[b]), int(cu_seqlens_q[b + 1])
        L, S = z - a, int(seqused_k[b])
        for t in range(L):
            lo, hi = first_visible_key(S, L, t, window_left), visible_keys(S, L, t)
            if lo >= hi:
                continue
            keys = np.arange(lo, hi)
            page = np.asarray(block_table[b])[keys // PAGE_SIZE]
            slot = keys % PAGE_SIZE
            for h in range(Hkv):
                ks = read_scales(k_scales[page, h])
                vs = read_scales(v_scales[page, h])
                K = k[page, slot, h] * ks[:, None]
                C = v[page, slot, h]
                rows = q[a + t, h * G:(h + 1) * G]
                x = scale * (rows @ K.T)
                d = 2.0 ** -8 * abs(scale) * (np.abs(rows) @ np.abs(K).T)
                if softcap:
                    d = d + 2.0 ** -11 * np.abs(x)
                x = softcapped(x, softcap)
                m = x.max(axis=1, keepdims=True)
                if sinks is not None:
                    m = np.maximum(m, sinks[h * G:(h + 1) * G, None])
                w = np.exp(x - m)
                den = w.sum(axis=1, keepdims=True)
                if sinks is not None:
                    den = den + np.exp(sinks[h * G:(h + 1) * G, None] - m)
                w /= den
                o = (w * vs) @ C
                dmax = d.max(axis=1, keepdims=True)
                part = (w * vs) @ np.abs(C)
                block = np.flatnonzero(np.diff(keys // BLOCK, prepend=-1))
                top, size = np.maximum.reduceat(w * vs, block, axis=1), np.add.reduceat(np.abs(C), block, axis=0)
                floor = 2.0 ** -22 * top @ size + 2.0 ** -115 * top.max(axis=1, keepdims=True) * size.sum(axis=0)
                with np.errstate(over="ignore"):
                    tol[a + t, h * G:(h + 1) * G] = part * (np.expm1(2 * dmax) + 2.0 ** -8 + 2 * len(keys) * 2.0 ** -24) \
                        + floor + 2.0 ** -8 * np.abs(o)
                out[a + t, h * G:(h + 1) * G] = o
    return out, tol
