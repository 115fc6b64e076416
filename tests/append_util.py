"""Helpers of the append tests: batches, the oracle on the same bytes, and the
comparison, with tolerances from the number formats."""
from __future__ import annotations

import ctypes

import numpy as np
import torch

import speculative_decoding_verify_split_gb300 as va
from oracle.append_fp64 import append_oracle, rotated
from oracle.attention_fp64 import decode_bf16, decode_e4m3fn

# A rounding to nearest is off by at most half a step: eps / 2 of the value
# (bf16 2^-8, e4m3 2^-4), or half the spacing of e4m3's subnormals, 2^-10
# codes. Before it stand fp32 operations: two products and a sum of a rotated
# column, each within 2^-24 of its own size, and a quotient, so at most
# 4 * 2^-24 of |x1| + |x2|.
HALF = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
FP32 = 4 * 2.0 ** -24


def descriptors(*tensors):
    """Arguments of the C calls: pointers to va_tensor, None for none."""
    return [None if t is None else ctypes.pointer(va.desc(t)) for t in tensors]


def rope_of(cos_sin, positions=None, interleaved=0):
    if cos_sin is None:
        return None
    c, p = descriptors(cos_sin, positions)
    return ctypes.pointer(va.VaRope(c, p, interleaved))


def raw(t):
    t = t.detach().cpu().contiguous()
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8).numpy()
    return t.view(torch.int16).numpy().view(np.uint16)


def decode(t):
    return decode_e4m3fn(raw(t)) if t.dtype == torch.float8_e4m3fn else decode_bf16(raw(t))


def table(positions, rot, base=10000.0):
    half = rot // 2
    ang = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([ang.cos(), ang.sin()], dim=1).float()


class Batch:
    """New tokens of a batch and a cache with garbage in it (CPU tensors)."""

    def __init__(self, q_lens, kv_lens, hq, hkv, kind, rot, seed, dim=256, tail=0, interleaved=False):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.interleaved, self.hkv, self.dim = kind, interleaved, hkv, dim
        T = sum(q_lens) + tail
        width = max([1] + [-(-s // 16) for s in kv_lens])
        need = [max(1, -(-s // 16)) for s in kv_lens]
        self.pages = sum(need) + 2
        perm = torch.randperm(self.pages, generator=g).to(torch.int32)
        bt = torch.full((len(q_lens), width), int(perm[-1]), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            bt[b, :n] = perm[at:at + n]
            at += n
        self.block_table = bt
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32)
        self.used = torch.tensor(kv_lens, dtype=torch.int32)
        size = torch.exp2(2 * torch.randn(T, 1, 1, generator=g))
        self.k = (size * torch.randn(T, hkv, dim, generator=g)).to(torch.bfloat16)
        self.v = (size * torch.randn(T, hkv, dim, generator=g)).to(torch.bfloat16)
        qd = dim if dim == 256 else 64
        self.q = torch.randn(T, hq, qd, generator=g).to(torch.bfloat16)
        self.cos_sin = table(max([1] + list(kv_lens)), rot) if rot else None
        dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        shape = (self.pages, 16, hkv, dim)
        self.caches = [(100 * torch.randn(shape, generator=g)).clamp(-448, 448).to(dt) for _ in range(2)]
        self.scales = [torch.exp2(torch.randint(-9, 2, (self.pages, hkv), generator=g).float()) for _ in range(2)] \
            if kind == "scaled" else [None, None]
        self.descales = [torch.tensor([0.07]), torch.tensor([0.031])] if kind == "e4m3" else [None, None]
        self.positions = None

    def rope_position(self, b, t, row):
        if self.positions is not None:
            return int(self.positions[row])
        L = int(self.cu[b + 1] - self.cu[b])
        return int(self.used[b]) - L + t

    def turned(self, x):
        """x [T, heads, dim] rotated in fp64 (rows behind the last sequence as they are)."""
        y = decode(x)
        for b in range(len(self.used)):
            a, z = int(self.cu[b]), int(self.cu[b + 1])
            for t in range(z - a):
                y[a + t] = rotated(y[a + t], None if self.cos_sin is None else self.cos_sin.numpy(),
                                   self.rope_position(b, t, a + t), self.interleaved)
        return y

    def placed(self):
        """[T] bool: tokens at a position >= 0 of some sequence."""
        m = np.zeros(self.k.shape[0], dtype=bool)
        for b in range(len(self.used)):
            a, z = int(self.cu[b]), int(self.cu[b + 1])
            m[a:z] = np.arange(z - a) + int(self.used[b]) - (z - a) >= 0
        return m


def expect(b, rows, which):
    before = decode(b.caches[which]) if b.kind == "scaled" else None
    return append_oracle(rows, b.block_table.numpy(), b.cu.numpy(), b.used.numpy(), b.pages, before,
                         None if b.scales[which] is None else b.scales[which].numpy(),
                         None if b.descales[which] is None else float(b.descales[which]),
                         limit=448.0 if b.kind != "bf16" else np.inf)


def pair_size(rows_raw):
    """An upper bound of |x1| + |x2| over a row's pairs: twice its largest |value|."""
    f = np.where(np.isfinite(rows_raw), np.abs(rows_raw), 0)
    return 2 * f.max(axis=-1, initial=0.0)


def check_store(before, after, want, scales_after, descale, size):
    """The cache after the call against the oracle's Store: bytes of slots that
    got nothing are unchanged; the others are within half a step of the value,
    plus fp32's part of ``size`` (the largest |x1| + |x2| of the new rows)."""
    untouched = ~(want.written | want.kept)
    assert (raw(after)[untouched] == raw(before)[untouched]).all(), "a slot that got nothing changed"
    got = decode(after)
    if want.scales is not None:
        s = scales_after.cpu().numpy().astype(np.float64)
        assert np.array_equal(s, want.scales, equal_nan=True), "page scales"
        step = np.clip(np.nan_to_num(s, nan=0.0), 2.0 ** -64, 2.0 ** 64)[:, None, :, None]
    else:
        step = 1.0 if descale is None else float(descale)
    got = got * step
    m = ~untouched
    half = HALF[after.dtype]
    tol = np.maximum(half * np.abs(want.value), 0 if after.dtype == torch.bfloat16 else 2.0 ** -10 * step) + FP32 * size
    g, w, tol = got[m], want.value[m], np.broadcast_to(tol, got.shape)[m]
    assert np.array_equal(np.isnan(g), np.isnan(w)), "NaN"
    fin = np.isfinite(w)
    assert np.array_equal(g[~fin & ~np.isnan(w)], w[~fin & ~np.isnan(w)]), "infinities"
    bad = np.abs(g[fin] - w[fin]) > tol[fin]
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} stored values off, worst {np.abs(g[fin] - w[fin]).max()}"


def check_rotated(before, after, want, placed):
    """q_out: rows with a position within bf16's half step, others as they were."""
    assert (raw(after)[~placed] == raw(before)[~placed]).all(), "a row without a position changed"
    g, w = decode(after)[placed], want[placed]
    tol = HALF[torch.bfloat16] * np.abs(w) + FP32 * pair_size(w)[..., None]
    assert (np.abs(g - w) <= tol).all(), f"worst {np.abs(g - w).max()}"


def gpu(x):
    return None if x is None else x.to("cuda")


def run_kv(b, stream=None, in_place=False):
    """append_kv on copies of the batch's tensors: (q_out before, q_out, caches, scales)."""
    caches, scales = [gpu(c) for c in b.caches], [gpu(s) for s in b.scales]
    q = gpu(b.q) if b.cos_sin is not None else None
    q_out = None if q is None else q if in_place else torch.full_like(q, 7.0)
    before = None if q is None else q_out.cpu()
    va.append_kv(gpu(b.k), gpu(b.v), caches[0], caches[1], gpu(b.block_table), gpu(b.cu), gpu(b.used), q=q, q_out=q_out,
                 cos_sin=gpu(b.cos_sin), positions=gpu(b.positions), interleaved=b.interleaved, k_descale=gpu(b.descales[0]),
                 v_descale=gpu(b.descales[1]), k_scales=scales[0], v_scales=scales[1], stream=stream)
    torch.cuda.synchronize()
    return before, q_out, caches, scales


def check_kv(b, **kw):
    before, q_out, caches, scales = run_kv(b, **kw)
    if q_out is not None:
        check_rotated(before, q_out, b.turned(b.q), b.placed())
    for which, x in ((0, b.turned(b.k)), (1, decode(b.v))):
        size = pair_size(decode(b.k if which == 0 else b.v)).max(initial=0.0)
        check_store(b.caches[which], caches[which], expect(b, x, which), scales[which], b.descales[which], size)
    return caches, scales


def run_mla(b, stream=None, fused=True):
    cache, scales = gpu(b.caches[0]), gpu(b.scales[0])
    row = gpu(b.k)[:, 0]
    lat, pe = (row[:, :512], row[:, 512:]) if fused else (row[:, :512].contiguous(), row[:, 512:].contiguous())
    q_pe = gpu(b.q) if b.cos_sin is not None else None
    full = torch.full((b.q.shape[0], b.q.shape[1], 576), 7.0, dtype=torch.bfloat16, device="cuda")
    q_out = None if q_pe is None else full[..., 512:]
    before = None if q_pe is None else q_out.cpu()
    va.append_mla(lat, pe, cache, gpu(b.block_table), gpu(b.cu), gpu(b.used), q_pe=q_pe, q_pe_out=q_out, cos_sin=gpu(b.cos_sin),
                  positions=gpu(b.positions), interleaved=b.interleaved, descale=gpu(b.descales[0]), scales=scales, stream=stream)
    torch.cuda.synchronize()
    assert (full[..., :512] == 7.0).all()
    return before, q_out, cache, scales


def check_mla(b, **kw):
    before, q_out, cache, scales = run_mla(b, **kw)
    if q_out is not None:
        check_rotated(before, q_out, b.turned(b.q), b.placed())
    x = decode(b.k)
    full, b_dim = b.k, x.copy()
    b_dim[..., 512:] = b.turned(full[..., 512:])
    size = pair_size(x).max(initial=0.0)
    check_store(b.caches[0], cache, expect(b, b_dim, 0), scales, b.descales[0], size)
    return cache, scales
