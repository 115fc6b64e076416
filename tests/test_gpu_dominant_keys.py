"""Rows whose softmax has dominant keys (an attention sink), on the GPU against
fp64, for e4m3 caches with one descale and with page scales, GQA and latent.

A dominant key is the case in which the other weights are small one by one and
carry the output together: here its own value is small and the others have a
common mean, so a kernel that loses the small weights loses the output.

Bound: the relative L2 error of every row is at most ROW = 2^-7 + 2^-9. A weight
is stored as two e4m3 terms, within 2^-8 of itself (the second term is within
2^-4 of a remainder of at most 2^-4), and the output is rounded to bf16 (2^-8);
2^-9 is left for the exponential, fp32 sums and what the terms flush: weights
below 2^-20 of the largest of the 32 keys that they share a scale with. The
logits here are exact in the kernels' operands: keys of 0 and 1, and the 8 bits
of a bf16 query as two e4m3 terms."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
ROW = 2.0 ** -7 + 2.0 ** -9
WEIGHTS = (0.3, 0.5, 0.8, 0.9)


class Case:
    """B sequences of S keys, L draft tokens, hq heads (one KV head), whose heads
    give `spikes` (key positions) WEIGHTS of the row together. Logits: the last
    column of q times that of K, 0 for the other keys."""

    def __init__(self, latent, S, hq, L=1, B=1, spikes=(0,), spike_scale=1.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.latent, self.S, self.L, self.B, self.hq = latent, S, L, B, hq
        dim, dv = (576, 512) if latent else (256, 256)
        per = -(-S // 16)
        n = B * per
        self.pages = n
        val = torch.randn(n * 16, dv, device="cuda", generator=g) + 1.0
        key = torch.zeros(n * 16, dim, device="cuda")
        where = torch.tensor([b * per * 16 + s for b in range(B) for s in spikes], device="cuda")
        val[where] = 0.0625
        key[where, dim - 1] = 1.0
        self.scales = torch.ones(n, 1, device="cuda")
        self.scales[where // 16] = spike_scale
        if latent:
            key[:, :512] = val
            self.cache = self._codes(key)
        else:
            self.k, self.v = key.view(n, 16, 1, dim).to(F8), self._codes(val)
        self.q = torch.zeros(B * L, hq, dim, device="cuda", dtype=torch.bfloat16)
        for h in range(hq):
            w = WEIGHTS[h % len(WEIGHTS)]
            self.q[:, h, dim - 1] = math.log(w / (1 - w) * (S - len(spikes)) / len(spikes))
        self.table = torch.randperm(n, device="cuda", generator=g).to(torch.int32).view(B, per)
        self._place()
        self.cu = (torch.arange(B + 1, device="cuda") * L).to(torch.int32)
        self.used = torch.full((B,), S, dtype=torch.int32, device="cuda")

    def _codes(self, x):
        x = x.view(self.pages, 16, 1, -1)
        return (x / self.scales[:, None, :, None]).to(F8)

    def _place(self):
        order = self.table.view(-1).long()

        def put(t):
            out = torch.zeros_like(t.view(torch.uint8) if t.dtype == F8 else t)
            out[order] = t.view(torch.uint8) if t.dtype == F8 else t
            return out.view(F8) if t.dtype == F8 else out

        if self.latent:
            self.cache = put(self.cache)
        else:
            self.k, self.v = put(self.k), put(self.v)
        self.scales = put(self.scales)

    def reference(self, paged, window_left=-1):
        """fp64; page scales if `paged`, else 1."""
        sc = self.scales.double() if paged else torch.ones_like(self.scales).double()
        one = torch.ones_like(sc)
        out = torch.zeros(self.B * self.L, self.hq, 512 if self.latent else 256, dtype=torch.float64, device="cuda")
        for b in range(self.B):
            pg = self.table[b].long()
            if self.latent:
                K = (self.cache[pg].double() * sc[pg][:, None, :, None]).view(-1, 576)[: self.S]
                V = K[:, :512]
            else:
                K = (self.k[pg].double() * one[pg][:, None, :, None]).view(-1, 256)[: self.S]
                V = (self.v[pg].double() * sc[pg][:, None, :, None]).view(-1, 256)[: self.S]
            for t in range(self.L):
                i = b * self.L + t
                hi = self.S - self.L + t + 1
                lo = max(0, hi - 1 - window_left) if window_left >= 0 else 0
                p = torch.softmax(self.q[i].double() @ K[lo:hi].T, dim=1)
                out[i] = p @ V[lo:hi]
        return out

    def call(self, paged, splits, window_left=-1):
        args = (self.table, self.cu, self.used, self.L, self.table.shape[1] * 16, 1.0)
        if self.latent:
            if paged:
                return va.verify_attn_mla_scaled(self.q, self.cache, self.scales, *args, num_splits=splits)
            ws = torch.zeros(va.mla_workspace_size(self.q, self.used, *args[3:5], splits) + 256, dtype=torch.uint8, device="cuda")
            return va.verify_attn_mla(self.q, self.cache, *args, workspace=ws, num_splits=splits)
        if paged:
            return va.verify_attn_scaled(self.q, self.k, self.v, torch.ones_like(self.scales), self.scales, *args, num_splits=splits,
                                         window_left=window_left)
        if window_left >= 0:
            ws = torch.zeros(va.workspace_size(self.q, self.k, self.used, *args[3:5], splits) + 256, dtype=torch.uint8, device="cuda")
            return va.verify_attn_opt(self.q, self.k, self.v, *args, window_left=window_left, workspace=ws, num_splits=splits)
        return va.verify_attn_ex(self.q, self.k, self.v, *args, num_splits=splits)

    def check(self, paged, splits, window_left=-1, skip=0):
        got = self.call(paged, splits, window_left).double()[..., skip:]
        ref = self.reference(paged, window_left)[..., skip:]
        err = ((got - ref).norm(dim=-1) / ref.norm(dim=-1)).cpu().numpy()
        assert np.isfinite(err).all() and err.max() <= ROW, f"rows' relative errors up to {err.max():.4f}: {err.max(axis=0).round(4)}"


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("S", [1025, 8192, 65531])
@pytest.mark.parametrize("splits", [0, 1, 10])
def test_a_sink(paged, latent, S, splits):
    Case(latent, S, 16, seed=S).check(paged, splits)


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("hq,L", [(4, 1), (16, 2), (16, 3), (16, 4)])
@pytest.mark.parametrize("at", [0, 700, 4090])
def test_where_the_sink_lies_and_rows(latent, hq, L, at):
    """In the first tile, in the middle, behind nearly all keys; 4 to 64 packed rows."""
    c = Case(latent, 4099, hq, L, B=2, spikes=(at,), seed=hq + L)
    for splits in (0, 1):
        c.check(True, splits)


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("every", [33, 128, 1000])
def test_many_dominant_keys(latent, every):
    """One key in `every`: each tile holds some, beside keys that count."""
    c = Case(latent, 16384, 16, spikes=tuple(range(7, 16384, every)), seed=every)
    for splits in (0, 1):
        c.check(True, splits)


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** -6, 32.0])
def test_a_sink_in_a_page_of_another_scale(latent, scale):
    """Its page's V scale is a sixty-fourth, or 32 times, of the others'."""
    for S in (4096, 16384):
        for splits in (0, 1):
            Case(latent, S, 16, spike_scale=scale, seed=3).check(True, splits)


@pytest.mark.parametrize("exponent", [8, 12, 20])
def test_a_page_of_large_values_in_one_column(exponent):
    """Equal logits; one page's V scale is 2^exponent of the others', for its values
    in column 0. The other columns come from the other pages."""
    for splits in (0, 1):
        c = Case(False, 4096, 16, seed=9)
        c.q.zero_()
        pg = int(c.table[0, 5])
        v = c.v.float()
        v[pg] = 0.0
        v[pg, :, :, 0] = 256.0
        c.v = v.to(F8)
        c.scales[pg] = 2.0 ** exponent
        c.check(True, splits, skip=1)


def test_a_sink_and_a_window():
    """The variant kernel: a window that holds the dominant key, and one that does not."""
    c = Case(False, 8192, 16, spikes=(3000,), seed=4)
    for paged in (True, False):
        for splits in (0, 1):
            for w in (6000, 1 << 20, 2000):
                c.check(paged, splits, window_left=w)


def test_a_sink_over_shards():
    """Context-parallel shards: the same rows through verify_attn_partial and the merge."""
    c = Case(False, 8192, 16, seed=6)
    parts = []
    half = 4096 // 16
    for i in range(2):
        parts.append(va.verify_attn_partial(c.q, c.k, c.v, c.table[:, i * half:(i + 1) * half].contiguous(), c.cu,
                                            torch.full_like(c.used, 4096), 1, 4096, 1.0,
                                            kv_extent=torch.full_like(c.used, 8192 - 4096 * i), num_splits=3))
    got = va.merge_partials(parts).double()
    ref = c.reference(False)
    err = (got - ref).norm(dim=-1) / ref.norm(dim=-1)
    assert err.max() <= ROW


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("hq,L", [(8, 1), (16, 2), (16, 4)])
@pytest.mark.parametrize("levels", [(0, 1, 2, 3, 4, 5), (5, 4, 3, 2, 1, 0), (2, 0, 4, 1, 5, 3), (0, 0, 6, 6, 0, 0)])
def test_levels_far_apart(latent, hq, L, levels):
    """Runs of 200 keys whose logits lie 40 log2 units apart: a row's reference
    moves where a higher run begins (the accumulators follow it), stays where a
    lower one does, and the highest run alone makes the output."""
    c = Case(latent, 1200, hq, L, B=2, seed=11)
    dim = 576 if latent else 256
    step = 40.0 / math.log2(math.e)
    c.q[..., dim - 1] = step
    key = torch.tensor(levels, device="cuda", dtype=torch.float32).repeat_interleave(200)
    k = c.cache if latent else c.k
    x = k.float()
    for b in range(c.B):
        pg, n = c.table[b].long(), c.S
        rows = x[pg].view(-1, dim)
        rows[:n, dim - 1] = key
        x[pg] = rows.view(len(pg), 16, 1, dim)
    if latent:
        c.cache = x.to(F8)
    else:
        c.k = x.to(F8)
    for paged in (True, False):
        for splits in (0, 1, 3):
            c.check(paged, splits)


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("gap", [40, 72, 110])
def test_value_scales_at_both_ends_of_their_range(latent, gap):
    """One key in a page of scale 2^64, `gap` log2 units above the others, whose
    pages' scale is 2^-64: weight times scale of the others falls to 2^-238 of the
    row's largest, and they must not count for more than they are."""
    c = Case(latent, 1000, 16, seed=12)
    dim = 576 if latent else 256
    c.scales.fill_(2.0 ** -64)
    c.scales[int(c.table[0, 0])] = 2.0 ** 64
    c.q[..., dim - 1] = gap / math.log2(math.e) * (2.0 ** -64 if latent else 1.0)
    for t in (c.cache,) if latent else (c.k, c.v):        # a value of the size of the others', nothing else on its page
        x = t.float()
        pg = int(c.table[0, 0])
        if t is not (None if latent else c.k):
            x[pg] = 0.0
            x[pg, 0, 0, :256] = 3.0
        if latent:
            x[pg, 0, 0, dim - 1] = 1.0
        t.copy_(x.to(F8))
    for splits in (0, 1, 3):
        c.check(True, splits)
