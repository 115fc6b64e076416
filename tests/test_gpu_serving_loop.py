"""The calls of a serving loop together: prompts in chunks (norms, rotation, append, chunk
attention), branches that share their parents' pages, pages of their own for what they write,
copies, drafts appended and verified, branches freed. Against the oracles at every step,
with the cache's own contents as they are then."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import decode, gpu, raw, table as angles
from chunk_util import Chunk, tolerance
from oracle import page_pool as pool

pytestmark = pytest.mark.gpu
I = torch.int32
HQ, HKV, SEQS, WIDTH, PAGES = 16, 2, 8, 24, 96


class Loop:
    def __init__(self, kind, seed):
        self.kind, self.g = kind, torch.Generator().manual_seed(seed)
        dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        nan = torch.full((PAGES, 16, HKV, 256), float("nan")).to(dt)      # what no one has written is not read
        self.caches = [nan.cuda(), nan.cuda()]
        self.scales = [torch.zeros(PAGES, HKV, device="cuda") for _ in range(2)] if kind == "scaled" else [None, None]
        self.descales = [torch.tensor([0.05], device="cuda"), torch.tensor([0.03], device="cuda")] if kind == "e4m3" else [None, None]
        self.table = torch.full((SEQS, WIDTH), -1, dtype=I, device="cuda")
        self.used, self.count = (torch.zeros(SEQS, dtype=I, device="cuda") for _ in range(2))
        self.refs = torch.zeros(PAGES, dtype=I, device="cuda")
        self.status = torch.zeros(1, dtype=I, device="cuda")
        self.host = [self.table.tolist(), [0] * SEQS, [0] * SEQS, [0] * PAGES]
        self.cos_sin = gpu(angles(WIDTH * 16, 64))
        self.norms = [(1 + 0.2 * torch.randn(256, generator=self.g)).to(torch.bfloat16).cuda() for _ in range(2)]
        self.pools = (self.table, self.used, self.count, self.refs)

    def step(self, add):
        """add[b] new tokens of each row: reserve, copy, append, attend."""
        new = torch.tensor(add, dtype=I, device="cuda")
        src, dst, room = va.reserve_pages(*self.pools, new, status=self.status)
        va.copy_pages(*self.caches, src, dst, k_scales=self.scales[0], v_scales=self.scales[1])
        self.used += new
        cu = torch.zeros(SEQS + 1, dtype=I, device="cuda")
        cu[1:] = torch.cumsum(new, 0)
        T = sum(add)
        q, k, v = ((torch.randn(T, h, 256, generator=self.g)).to(torch.bfloat16).cuda() for h in (HQ, HKV, HKV))
        kw = dict(k_descale=self.descales[0], v_descale=self.descales[1], k_scales=self.scales[0], v_scales=self.scales[1])
        va.append_kv(k, v, *self.caches, self.table, cu, self.used, q=q, q_out=q, cos_sin=self.cos_sin, q_norm=self.norms[0],
                     k_norm=self.norms[1], **kw)
        out = va.verify_attn_chunk(q, *self.caches, self.table, cu, self.used, 0.0625, **kw)
        torch.cuda.synchronize()
        bits, *want = pool.reserve(*self.host, add)
        assert bits == 0 and int(self.status) == 0
        assert [x.tolist() for x in (src, dst, room)] == want
        self.host[1] = [u + a for u, a in zip(self.host[1], add)]
        self.same()
        b = self.batch(q, cu)
        ref, size = b.expect()
        tol = tolerance(b, ref, size)
        assert (np.abs(decode(out) - ref) <= tol).all()
        assert va.last_device_error() == 0
        return b, q, cu, ref, tol

    def batch(self, q, cu):
        b = Chunk.__new__(Chunk)
        b.kind, b.hq, b.hkv, b.scale = self.kind, HQ, HKV, 0.0625
        b.q, b.cu, b.used, b.table = q.cpu(), cu.cpu(), self.used.cpu(), self.table.cpu().clamp(min=0)
        b.caches = [c.cpu() for c in self.caches]
        b.scales = [None if s is None else s.cpu() for s in self.scales]
        b.descales = [None if d is None else d.cpu() for d in self.descales]
        return b

    def same(self):
        assert [x.tolist() for x in self.pools] == self.host


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "scaled"])
def test_prompts_branches_and_drafts(kind):
    w = Loop(kind, 41)
    w.step([100, 37, 1, 0, 0, 0, 0, 0])          # prompts,
    w.step([29, 64, 130, 0, 0, 0, 0, 0])         # and further pieces of them
    parents, children = [0, 0, 1, 2, 2], [3, 4, 5, 6, 7]
    va.fork_pages(*w.pools, torch.tensor(parents, dtype=I, device="cuda"), torch.tensor(children, dtype=I, device="cuda"), status=w.status)
    assert pool.fork(*w.host, parents, children) == 0
    before = [c.clone() for c in w.caches]
    shared = [[w.host[0][p][i] for i in range(w.host[1][p] // 16)] for p in range(3)]
    b, q, cu, ref, tol = w.step([0, 0, 0, 4, 3, 2, 1, 4])
    for pages in shared:                         # full pages are the parents' still, with their contents
        for c, x in zip(w.caches, before):
            assert (raw(c)[pages] == raw(x)[pages]).all()
    # the verify kernel over the same branches
    a = (w.table, cu, w.used, 4, WIDTH * 16, 0.0625)
    if kind == "scaled":
        out = va.verify_attn_scaled(q, *w.caches, *w.scales, *a)
    else:
        out = va.verify_attn(q, *w.caches, *a, *w.descales)
    torch.cuda.synchronize()
    assert (np.abs(decode(out) - ref) <= 1e-2 + 1e-2 * np.abs(ref)).all()
    # the losing branches go; parents write on, over pages of their own again
    va.free_pages(*w.pools, torch.tensor([3, 5, 6], dtype=I, device="cuda"), status=w.status)
    assert pool.free(*w.host, [3, 5, 6]) == 0
    w.step([5, 16, 1, 0, 20, 0, 0, 3])
    va.free_pages(*w.pools, torch.tensor(list(range(SEQS)), dtype=I, device="cuda"), status=w.status)
    assert pool.free(*w.host, list(range(SEQS))) == 0
    w.same()
    assert sum(w.refs.tolist()) == 0
