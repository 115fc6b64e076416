"""Chunk attention (verify_attn_chunk) in fp64, row by row from its definition."""
from __future__ import annotations

import numpy as np

PAGE = 16


def chunk_oracle(q, k, v, table, cu, used, scale, window_left=-1, first_tokens=0, softcap=0.0, sinks=None):
    """q [T, Hq, D]; k, v [pages, 16, Hkv, D]: the caches' values (decoded,
    descaled), all fp64. Returns (out [T, Hq, D], size [T, Hq, D]): the attention
    and sum_j p_j |V_j|, what a relative error of the weights and of P V acts on.
    Rows outside the sequences stay NaN in ``out``."""
    T, hq, D = q.shape
    hkv = k.shape[2]
    group = hq // hkv
    out = np.full((T, hq, D), np.nan)
    size = np.zeros((T, hq, D))
    for b in range(len(used)):
        a, z = int(cu[b]), int(cu[b + 1])
        L, S = z - a, int(used[b])
        pages = table[b, :-(-S // PAGE)]
        for h in range(hkv):
            kk = k[pages, :, h].reshape(-1, D)[:S]
            vv = v[pages, :, h].reshape(-1, D)[:S]
            for t in range(L):
                i = S - L + t
                j = np.arange(max(0, i + 1))
                if window_left >= 0:
                    j = j[(j >= i - window_left) | (j < first_tokens)]
                for g in range(h * group, (h + 1) * group):
                    if len(j) == 0:
                        out[a + t, g] = 0.0
                        continue
                    s = scale * (kk[j] @ q[a + t, g])
                    if softcap > 0:
                        s = softcap * np.tanh(s / softcap)
                    top = s.max()
                    p = np.exp(s - top)
                    den = p.sum() + (np.exp(sinks[g] - top) if sinks is not None else 0.0)
                    out[a + t, g] = p @ vv[j] / den
                    size[a + t, g] = p @ np.abs(vv[j]) / den
    return out, size
