"""free_pages, fork_pages, reserve_pages and copy_pages on the GPU: exactly what
the oracle does, through random rounds, in every corner of a pool."""
import random

import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import raw
from oracle import page_pool as pool

pytestmark = pytest.mark.gpu
I = torch.int32


class Both:
    """A pool on the GPU and its twin on the host."""

    def __init__(self, seqs, width, pages, strided=False):
        self.table = torch.full((seqs, 2 * width), -7, dtype=I, device="cuda")[:, ::2] if strided else \
            torch.full((seqs, width), -7, dtype=I, device="cuda")
        self.used, self.count = (torch.zeros(seqs, dtype=I, device="cuda") for _ in range(2))
        self.refs = torch.zeros(pages, dtype=I, device="cuda")
        self.status = torch.zeros(1, dtype=I, device="cuda")
        self.host = [self.table.tolist(), [0] * seqs, [0] * seqs, [0] * pages]
        self.bits = 0

    def pools(self):
        return self.table, self.used, self.count, self.refs

    def set(self, **kw):
        """Sets arrays on both sides."""
        for k, v in kw.items():
            getattr(self, k).copy_(torch.tensor(v, dtype=I))
            self.host[["table", "used", "count", "refs"].index(k)] = [list(x) for x in v] if k == "table" else list(v)

    def same(self):
        torch.cuda.synchronize()
        assert self.table.tolist() == self.host[0]
        assert self.used.tolist() == self.host[1]
        assert self.count.tolist() == self.host[2]
        assert self.refs.tolist() == self.host[3]
        assert int(self.status) == self.bits

    def free(self, seqs):
        va.free_pages(*self.pools(), torch.tensor(seqs, dtype=I, device="cuda"), status=self.status)
        self.bits |= pool.free(*self.host, seqs)
        self.same()

    def fork(self, parents, children):
        va.fork_pages(*self.pools(), torch.tensor(parents, dtype=I, device="cuda"), torch.tensor(children, dtype=I, device="cuda"),
                      status=self.status)
        self.bits |= pool.fork(*self.host, parents, children)
        self.same()

    def reserve(self, add):
        got = va.reserve_pages(*self.pools(), torch.tensor(add, dtype=I, device="cuda"), status=self.status)
        bits, *want = pool.reserve(*self.host, add)
        self.bits |= bits
        self.same()
        assert [x.tolist() for x in got] == want
        return want

    def write(self, add, room):
        """The tokens that were reserved for are there now."""
        used = [u + max(0, a) if r >= u + a else u for u, a, r in zip(self.host[1], add, room)]
        self.set(used=used)


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("seqs,width,pages,most", [(7, 9, 30, 20), (40, 12, 200, 60), (3, 70, 130, 900), (300, 5, 1100, 20)])
def test_rounds(seed, seqs, width, pages, most):
    r = random.Random(seed)
    b = Both(seqs, width, pages, strided=seed % 3 == 0)
    for _ in range(8):
        add = [r.choice([0, -3, 1, 4, 16, r.randrange(most)]) for _ in range(seqs)]
        src, dst, room = b.reserve(add)
        b.write(add, room)
        b.free([r.randrange(seqs) for _ in range(r.randrange(1, 1 + seqs // 3 + 1))])
        parents = [r.randrange(seqs) for _ in range(r.randrange(1, 2 + seqs // 2))]
        children = [r.randrange(-1, seqs + 1) if r.random() < 0.1 else r.randrange(seqs) for _ in parents]
        b.fork(parents, children)
        b.set(used=[max(0, u - r.choice([0, 0, 1, 5, 40])) for u in b.host[1]])   # rejected tokens


@pytest.mark.parametrize("pages", [1, 31, 32, 33, 255, 256, 257, 8192, 8193, 70001])
def test_pools_of_any_size(pages):
    """All pages but a few, through the pool's last word."""
    b = Both(3, -(-pages // 2) + 1, pages)
    half = pages // 2
    b.reserve([16 * half, 0, 16 * (pages - half)])
    assert b.refs.tolist() == [1] * pages
    b.reserve([0, 1, 0])                           # nothing left
    assert b.bits == va.PG_NO_PAGES
    b.free([2])
    b.reserve([0, 16 * (pages - half), 0])


def test_sequences_get_all_or_none_in_order():
    b = Both(5, 8, 10)
    b.reserve([64, 48, 80, 16, 0])                 # 4 + 3 fit, 5 do not, and so not the 1 behind
    assert b.count.tolist() == [4, 3, 0, 0, 0] and b.bits == va.PG_NO_PAGES
    b.reserve([0, 0, 0, 16, 0])
    assert b.count.tolist() == [4, 3, 0, 1, 0]


def test_shared_pages_are_replaced_where_they_are_written():
    b = Both(4, 8, 32)
    src, dst, room = b.reserve([40, 0, 0, 0])
    b.write([40, 0, 0, 0], room)
    b.fork([0, 0], [1, 2])
    assert b.refs.tolist()[:3] == [3, 3, 3]
    src, dst, room = b.reserve([0, 4, 20, 0])      # two candidates write on; the prompt rests
    assert src == [-1, 2, 2, -1] and dst == [-1, 3, 4, -1] and b.refs.tolist()[:7] == [3, 3, 1, 1, 1, 1, 0]   # 60 tokens: four pages
    b.free([1, 2])
    assert b.refs.tolist()[:6] == [1, 1, 1, 0, 0, 0]
    b.set(used=[20, 0, 0, 0])                      # tokens rejected across a page's border
    b.fork([0], [3])
    b.set(used=[17, 0, 0, 20])
    b.reserve([40, 0, 0, 1])                       # its second page is shared, its third its own
    b.set(used=[16, 0, 0, 16])
    b.reserve([1, 0, 0, 1])                        # at a border nothing holds tokens: no copy


def test_both_rows_of_a_page_write():
    """Each gets a page of its own; the shared one becomes free behind the call."""
    b = Both(2, 4, 8)
    *_, room = b.reserve([10, 0])
    b.write([10, 0], room)
    b.fork([0], [1])
    src, dst, _ = b.reserve([1, 1])
    assert src == [0, 0] and dst == [1, 2] and b.refs.tolist() == [0, 1, 1, 0, 0, 0, 0, 0]


def test_bad_arguments_are_reported_and_left():
    b = Both(4, 4, 16)
    *_, room = b.reserve([20, 20, 0, 0])
    b.write([20, 20, 0, 0], room)
    b.free([9, -1, 1 << 30])
    assert b.bits == va.PG_BAD_SEQ
    b.fork([0, 0, 0, 7], [1, 2, 2, 3])             # in use, fine, twice, no such parent
    b.fork([0, 3, 1], [3, 0, 1])                   # children that are parents
    assert b.bits == va.PG_BAD_SEQ | va.PG_IN_USE
    b.reserve([0, 1000, 0, 0])
    assert b.bits & va.PG_ROW_FULL
    b.set(count=[1, 2, 2, 0])                      # fewer pages than tokens
    b.fork([0], [3])
    assert b.bits & va.PG_BAD_TABLE
    b.set(count=[2, 2, 2, 0])


@pytest.mark.parametrize("entry", [-1, 16, -3, 1 << 30])
def test_pages_outside_the_pool(entry):
    b = Both(2, 4, 16)
    *_, room = b.reserve([20, 20])
    b.write([20, 20], room)
    t = [list(x) for x in b.host[0]]
    t[0][1] = entry
    b.set(table=t)
    b.reserve([4, 4])
    assert b.bits == va.PG_BAD_TABLE
    b.free([0, 1])


@pytest.mark.parametrize("counts", [[-1, 2], [9, 2]])
def test_counts_outside_the_row(counts):
    b = Both(2, 4, 16)
    *_, room = b.reserve([20, 20])
    b.write([20, 20], room)
    b.set(count=counts)
    b.reserve([4, 4])
    assert b.bits & va.PG_BAD_TABLE


def test_a_page_freed_too_often():
    b = Both(3, 2, 4)
    b.set(table=[[1, 0], [1, 0], [1, 0]], count=[1, 1, 1], used=[3, 3, 3], refs=[0, 1, 0, 0])
    b.free([0, 1, 2])
    assert b.bits == va.PG_BAD_TABLE and b.refs.tolist() == [0, 0, 0, 0]


def test_captured_round_on_a_stream():
    """Free, fork and reserve replayed: the pool goes round as it does eagerly."""
    b = Both(6, 20, 100)
    add = [100, 33, 0, 0, 0, 0]
    *_, room = b.reserve(add)
    b.write(add, room)
    lists = [torch.tensor(x, dtype=I, device="cuda") for x in ([2, 3, 4, 5], [0, 0, 1, 1], [0, 0, 5, 5, 40, 7])]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        va.free_pages(*b.pools(), lists[0], status=b.status)
        va.fork_pages(*b.pools(), lists[1], lists[0], status=b.status)
        out = va.reserve_pages(*b.pools(), lists[2], status=b.status)
    for _ in range(3):
        g.replay()
        b.bits |= pool.free(*b.host, [2, 3, 4, 5]) | pool.fork(*b.host, [0, 0, 1, 1], [2, 3, 4, 5])
        bits, *want = pool.reserve(*b.host, [0, 0, 5, 5, 40, 7])
        b.bits |= bits
        b.same()
        assert [x.tolist() for x in out] == want


# ---- copies ------------------------------------------------------------------------------


def cache(pages, heads, dim, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = pages * 16 * heads * dim * dtype.itemsize
    return torch.randint(0, 256, (n,), dtype=torch.uint8, generator=g).view(dtype).reshape(pages, 16, heads, dim)


def check_copy(k, v, ks, vs, src, dst, **kw):
    on = [None if x is None else x.cuda() if not callable(x) else x() for x in (k, v, ks, vs)]
    va.copy_pages(on[0], on[1], torch.tensor(src, dtype=I, device="cuda"), torch.tensor(dst, dtype=I, device="cuda"), k_scales=on[2],
                  v_scales=on[3], **kw)
    torch.cuda.synchronize()
    for before, after in zip((k, v, ks, vs), on):
        if before is None:
            continue
        want = before.clone()
        w = want.view(torch.uint8) if want.dtype == torch.float8_e4m3fn else want.view(torch.int16) if want.dtype == torch.bfloat16 else want
        for a, z in zip(src, dst):
            if 0 <= a < len(w) and 0 <= z < len(w):
                w[z] = w[a].clone()
        if want.dtype == torch.float32:
            assert torch.equal(want, after.cpu())
        else:
            assert (raw(want) == raw(after)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("heads,dim", [(1, 256), (2, 256), (3, 256), (8, 256), (1, 576), (5, 64), (33, 256)])
def test_copy(dtype, heads, dim):
    k, v = (cache(40, heads, dim, dtype, 3 + i) for i in range(2))
    src, dst = [0, 5, 39, 5, -1, 7, 40, 8, 3], [1, 9, 2, 38, 4, -1, 6, 8, 1 << 30]
    check_copy(k, v, None, None, src, dst)
    check_copy(k, None, None, None, src, dst)
    if dtype == torch.float8_e4m3fn:
        ks, vs = torch.rand(40, heads), torch.rand(40, heads)
        check_copy(k, v, ks, vs, src, dst)
        check_copy(k, None, ks, None, src, dst)


def test_copy_many_and_on_a_stream():
    k, v = (cache(700, 2, 256, torch.float8_e4m3fn, i) for i in range(2))
    ks, vs = torch.rand(700, 2), torch.rand(700, 2)
    perm = torch.randperm(700, generator=torch.Generator().manual_seed(1)).tolist()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check_copy(k, v, ks, vs, perm[:350], perm[350:], stream=s)


def test_copy_of_interleaved_caches_and_strided_heads():
    """K and V as views of one tensor, and a cache of every other head: the rest stays."""
    both = cache(20, 4, 512, torch.bfloat16, 5)
    on = both.cuda()
    k, v = on[:, :, ::2, :256], on[:, :, ::2, 256:]
    va.copy_pages(k, v, torch.tensor([3, 4], dtype=I, device="cuda"), torch.tensor([10, 11], dtype=I, device="cuda"))
    torch.cuda.synchronize()
    want = both.view(torch.int16).clone()
    want[10, :, ::2], want[11, :, ::2] = want[3, :, ::2].clone(), want[4, :, ::2].clone()
    assert (raw(on) == want.numpy().view("uint16")).all()
