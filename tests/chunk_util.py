"""Helpers of the chunk attention tests: batches with garbage where nothing may
be read, and the comparison, with a bound from the number formats."""
from __future__ import annotations

import numpy as np
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import decode, gpu
from oracle.chunk_fp64 import chunk_oracle

PAGE = 16


class Chunk:
    """A batch of new tokens over a paged cache (CPU tensors). Pages of the pool
    that no sequence uses, and slots behind a sequence's last token, hold NaN."""

    def __init__(self, q_lens, kv_lens, hq, hkv, kind, seed, tail=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.hq, self.hkv = kind, hq, hkv
        T = sum(q_lens) + tail
        need = [-(-s // PAGE) for s in kv_lens]
        width = max([1] + need)
        self.pages = sum(need) + 3
        perm = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(q_lens), width), int(perm[-1]), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32)
        self.used = torch.tensor(kv_lens, dtype=torch.int32)
        self.q = (spread * torch.randn(T, hq, 256, generator=g)).to(torch.bfloat16)
        self.scale = 256 ** -0.5
        dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        self.caches = []
        for _ in range(2):
            x = torch.randn(self.pages, PAGE, hkv, 256, generator=g)
            if kind != "bf16":
                x *= 20
            free = torch.ones(self.pages, PAGE, dtype=torch.bool)
            for b, s in enumerate(kv_lens):
                for p in range(-(-s // PAGE)):
                    free[int(self.table[b, p]), :min(PAGE, s - p * PAGE)] = False
            x[free] = float("nan")
            self.caches.append(x.to(dt))
        self.scales = [torch.exp2(torch.randint(-6, -2, (self.pages, hkv), generator=g).float()) for _ in range(2)] \
            if kind == "scaled" else [None, None]
        self.descales = [torch.tensor([0.05]), torch.tensor([0.03])] if kind == "e4m3" else [None, None]
        self.sinks = 2 * torch.randn(hq, generator=g)

    def values(self, i):
        x = np.nan_to_num(decode(self.caches[i]))
        if self.scales[i] is not None:
            s = np.clip(np.nan_to_num(self.scales[i].numpy().astype(np.float64), nan=0.0), 2.0 ** -64, 2.0 ** 64)
            x = x * s[:, None, :, None]
        if self.descales[i] is not None:
            x = x * float(self.descales[i])
        return x

    def expect(self, sinks=False, **kw):
        return chunk_oracle(decode(self.q), self.values(0), self.values(1), self.table.numpy(), self.cu.numpy(), self.used.numpy(),
                            self.scale, sinks=self.sinks.numpy().astype(np.float64) if sinks else None, **kw)

    def args(self):
        return [gpu(x) for x in (self.q, self.caches[0], self.caches[1], self.table, self.cu, self.used)]

    def run(self, sinks=False, out=None, **kw):
        out = torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        va.verify_attn_chunk(*self.args(), self.scale, k_descale=gpu(self.descales[0]), v_descale=gpu(self.descales[1]),
                             k_scales=gpu(self.scales[0]), v_scales=gpu(self.scales[1]), out=out,
                             sinks=gpu(self.sinks) if sinks else None, **kw)
        torch.cuda.synchronize()
        assert va.last_device_error() == 0
        return out


# What the output may be off by, for a row o = sum_j p_j V_j with sum p = 1:
#  * its rounding to bf16, 2^-8 of |o|;
#  * each p_j to the weights' type: 2^-8 of it (bf16), so sum_j p_j |V_j| 2^-8;
#    e4m3 caches take f16, 2^-11, with a floor of 2^-25 2^-7 2^8 of the largest
#    weight for each of n keys, at most n 2^-24 max|V| (part of `small`);
#  * the logits: sums of 256 products in fp32, within 256 2^-24 sum|q_d k_d| |scale|
#    of theirs, the exponents' fp32 arithmetic within 2^-22 of |s| log2(e), and the
#    SFU's 2^x within 2^-22: a relative error of each weight, numerator and
#    normaliser, so twice sum_j p_j |V_j| of it.
def tolerance(b, want, size, softcap=0.0):
    half = 2.0 ** -8 if b.kind == "bf16" else 2.0 ** -11
    q, k = np.abs(decode(b.q)), np.abs(b.values(0))
    bound = abs(b.scale) * q.sum(axis=2).max(initial=0.0) * k.max(initial=0.0)  # of |s|, and of sum|q_d k_d| |scale|
    logit = 256 * 2.0 ** -24 * bound + 2.0 ** -21 * 1.45 * bound + 2.0 ** -21
    if b.kind != "bf16":
        # q as two e4m3 terms of q 2^e, the row's largest in [2^7, 2^8): the second is
        # exact, or off by half of e4m3's smallest step, 2^-10: 2^-17 of the row's largest
        logit += abs(b.scale) * 2.0 ** -17 * q.max(initial=0.0) * k.sum(axis=3).max(initial=0.0)
    if softcap:
        # tanh by 2^x and a quotient: 2^-20 of it and of 1, times the cap
        logit += 2.0 ** -20 * softcap
    small = 2.0 ** -24 * float(b.used.max()) * np.abs(b.values(1)).max(initial=0.0) if b.kind != "bf16" else 0.0
    return 2.0 ** -8 * np.abs(want) + (half + 2 * logit) * size + small + 1e-30


def check(b, sinks=False, run_kw=None, **kw):
    want, size = b.expect(sinks=sinks, **kw)
    out = b.run(sinks=sinks, **kw, **(run_kw or {}))
    got = decode(out)
    inside = ~np.isnan(want).any(axis=(1, 2))
    assert (got[~inside] == 7.0).all(), "a row behind the last sequence changed"
    tol = tolerance(b, want, size, kw.get("softcap", 0.0))[inside]
    err = np.abs(got - want)[inside]
    assert np.isfinite(got[inside]).all(), "NaN or infinity in the output"
    bad = err > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outputs off, worst {err.max()} where {tol.flat[err.argmax()]} is allowed"
    return out
