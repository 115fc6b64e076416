"""verify_attn_chunk against the fp64 oracle: row tiles and key tiles that end
anywhere, every cache type, windows with first tokens, shares of the work."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import decode, gpu
from chunk_util import Chunk, check, tolerance

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "scaled"]


@pytest.mark.parametrize("kind", KINDS)
def test_one_token(kind):
    check(Chunk([1], [1], 1, 1, kind, 0))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv", [
    ([128], [128], 1, 1),            # one CTA's rows, one key tile
    ([256], [256], 1, 1),            # a pair's rows
    ([257], [300], 1, 1),            # one row more
    ([16], [1024], 16, 1),
    ([17, 40, 1], [200, 391, 129], 16, 1),
    ([3, 0, 70, 5], [3, 50, 70, 2000], 8, 2),
    ([33], [160], 3, 1),             # heads that do not divide a row tile
    ([90], [91], 5, 1),
    ([20, 31], [31, 47], 20, 4),
    ([5, 7], [3, 7], 4, 1),          # tokens before position 0 see nothing
    ([4], [0], 2, 1),                # nothing cached at all
])
def test_shapes(q_lens, kv_lens, hq, hkv, kind):
    check(Chunk(q_lens, kv_lens, hq, hkv, kind, sum(kv_lens) + hq, tail=2))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [0, 1, 2, 5, 64])
def test_shares(splits, kind):
    check(Chunk([20, 1, 33], [900, 700, 33], 8, 1, kind, 11), run_kw=dict(num_splits=splits))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,first", [(0, 0), (0, 1), (5, 4), (63, 0), (127, 130), (200, 16), (500, 3), (1 << 30, 7), (31, 2000)])
def test_windows_and_first_tokens(window, first, kind):
    check(Chunk([40, 1, 7], [700, 513, 7], 4, 1, kind, window % 97 + first), window_left=window, first_tokens=first)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [0, 1, 7])
def test_softcap_and_sinks(kind, splits):
    b = Chunk([20, 2], [300, 400], 8, 2, kind, 3, spread=4.0)
    check(b, sinks=True, softcap=15.0, run_kw=dict(num_splits=splits))
    check(b, sinks=True, run_kw=dict(num_splits=splits))
    check(b, sinks=True, softcap=8.0, window_left=100, first_tokens=4, run_kw=dict(num_splits=splits))


# ---- layouts, streams, graphs, what no test above reaches ------------------------------------


@pytest.mark.parametrize("kind", KINDS)
def test_strided_views(kind):
    """q a view of a wider projection, out of a wider buffer, K and V interleaved, a
    transposed block table, scales as one tensor."""
    b = Chunk([20, 9], [150, 64], 6, 2, kind, 5)
    want, size = b.expect()
    wide = torch.zeros(29, 10, 256, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:8] = gpu(b.q)
    buf = torch.full((29, 9, 264), 7.0, dtype=torch.bfloat16, device="cuda")
    both = torch.stack([gpu(c).view(torch.uint8 if kind != "bf16" else torch.int16) for c in b.caches], dim=3)
    both = both.view(b.caches[0].dtype)
    table = gpu(b.table).t().contiguous().t()
    sc = [None, None] if b.scales[0] is None else list(torch.stack([gpu(s) for s in b.scales], dim=2).unbind(2))
    va.verify_attn_chunk(wide[:, 2:8], both[:, :, :, 0], both[:, :, :, 1], table, gpu(b.cu), gpu(b.used), b.scale, k_descale=gpu(b.descales[0]),
                         v_descale=gpu(b.descales[1]), k_scales=sc[0], v_scales=sc[1], out=buf[:, 1:7, :256])
    torch.cuda.synchronize()
    got = decode(buf[:, 1:7, :256])
    assert (np.abs(got - want) <= tolerance(b, want, size)).all()
    rest = buf.clone()
    rest[:, 1:7, :256] = 7.0
    assert (rest == 7.0).all()


@pytest.mark.parametrize("scale", [0.3, -0.0625, 0.0])
@pytest.mark.parametrize("kind", KINDS)
def test_scales_of_either_sign(kind, scale):
    b = Chunk([9, 3], [140, 77], 4, 2, kind, 8)
    b.scale = scale
    check(b)
    check(b, softcap=5.0)


@pytest.mark.parametrize("kind", KINDS)
def test_rising_and_dominant_keys(kind):
    """References that move at every tile, and one key that outweighs all others."""
    b = Chunk([6], [1300], 4, 1, kind, 12, tail=0)
    k = torch.zeros(1312, 256)
    k[:, 0] = torch.linspace(0, 40, 1312)
    k[777, 0] = 44
    b.q.zero_()
    b.q[..., 0] = torch.tensor([16.0, 8.0, 1.0, -4.0])
    for p in range(82):
        page = int(b.table[0, p])
        b.caches[0][page, :, 0] = k[16 * p:16 * p + 16].to(b.caches[0].dtype)
    if b.scales[0] is not None:
        b.scales[0].fill_(1.0)
    if b.descales[0] is not None:
        b.descales[0].fill_(1.0)
    check(b)
    check(b, run_kw=dict(num_splits=5))


@pytest.mark.parametrize("kind", KINDS)
def test_unmapped_pages_of_a_window(kind):
    """Pages before every window and behind the first tokens need not be mapped."""
    b = Chunk([30], [900], 4, 1, kind, 21)
    want, size = b.expect(window_left=100, first_tokens=20)
    lo = (900 - 30 - 100) // 16
    b.table[0, 2:lo] = torch.tensor([-1, 1 << 30] * lo)[:lo - 2]
    out = b.run(window_left=100, first_tokens=20)
    assert (np.abs(decode(out) - want) <= tolerance(b, want, size)).all()


@pytest.mark.parametrize("kind", KINDS)
def test_nan_keys_that_nobody_sees(kind):
    """NaN in keys and values behind the last token (every batch here has them), and in keys
    of pages of the sequence that a window hides from every row."""
    b = Chunk([5], [700], 4, 1, kind, 22)
    page = int(b.table[0, 3])
    b.caches[0][page] = torch.full((16, 1, 256), float("nan")).to(b.caches[0].dtype)
    b.caches[1][page] = torch.full((16, 1, 256), float("nan")).to(b.caches[1].dtype)
    want, size = b.expect(window_left=200)
    out = b.run(window_left=200)
    assert (np.abs(decode(out) - want) <= tolerance(b, want, size)).all()


def test_nan_that_is_seen_shows():
    b = Chunk([4, 4], [40, 50], 2, 1, "bf16", 23)
    b.caches[0][int(b.table[0, 0]), 3] = float("nan")
    out = decode(b.run())
    assert np.isnan(out[:4]).all() and np.isfinite(out[4:]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_and_lengths_stay_inside(kind):
    """Page ids outside the cache, lengths past the table, prefix sums out of order: no access
    leaves the tensors, other sequences are right."""
    b = Chunk([20, 20, 20], [300, 300, 300], 4, 1, kind, 24)
    want, size = b.expect()
    b.table[1, 2] = 1 << 30
    b.table[1, 3] = -7
    b.used[1] = 100000
    out = decode(b.run())
    for rows in (slice(0, 20), slice(40, 60)):
        assert (np.abs(out - want) <= tolerance(b, want, size))[rows].all()
    b.cu = torch.tensor([0, 20, 10, 1000], dtype=torch.int32)
    b.run()


@pytest.mark.parametrize("kind", KINDS)
def test_empty_batches_and_caches(kind):
    b = Chunk([0, 0], [30, 0], 4, 1, kind, 25, tail=3)
    assert (b.run() == 7.0).all()
    b = Chunk([3], [0], 4, 1, kind, 26)
    b.caches = [c[:0] for c in b.caches]
    b.scales = [None if s is None else s[:0] for s in b.scales]
    assert (b.run() == 0.0).all()


def test_many_sequences():
    """More sequences than a CTA has threads, most without tokens."""
    q = [(i * 7) % 3 if i % 5 == 0 else 0 for i in range(1100)]
    kv = [max(n, (i * 13) % 40) for i, n in enumerate(q)]
    check(Chunk(q, kv, 2, 1, "bf16", 27))


@pytest.mark.parametrize("kind", KINDS)
def test_graph_and_other_stream_give_the_same_bits(kind):
    b = Chunk([33, 2], [500, 300], 8, 2, kind, 28)
    a = b.args()
    kw = dict(k_descale=gpu(b.descales[0]), v_descale=gpu(b.descales[1]), k_scales=gpu(b.scales[0]), v_scales=gpu(b.scales[1]))
    eager = va.verify_attn_chunk(*a, b.scale, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = va.verify_attn_chunk(*a, b.scale, stream=s, **kw)
    ws = torch.zeros(va.chunk_workspace_size(), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    outs = [torch.zeros_like(eager) for _ in range(3)]
    graphs = []
    for o, w in zip(outs, (None, None, ws)):          # two graphs with workspaces of their own, one with the caller's
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            va.verify_attn_chunk(*a, b.scale, out=o, workspace=w, **kw)
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(eager, x) for x in [side, *outs])
    assert va.workspace_status(ws) == 0 and va.last_device_error() == 0


def test_library_workspace_is_refused_during_capture():
    b = Chunk([3], [40], 2, 1, "bf16", 29)
    lib, held = va.library(), b.args()                # (a descriptor keeps no tensor alive)
    a = [va.desc(x) for x in held]
    out = torch.zeros(b.q.shape, dtype=torch.bfloat16, device="cuda")
    d = va.desc(out)
    import ctypes
    r = [ctypes.byref(x) for x in a]

    def call(stream):
        return lib.verify_attn_chunk(r[0], r[1], r[2], None, None, r[3], r[4], r[5], b.scale, None, None, ctypes.byref(d), None, 0, None, 0, 0,
                                     ctypes.c_void_p(stream))

    assert call(torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    want, size = b.expect()
    assert (np.abs(decode(out) - want) <= tolerance(b, want, size)).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        torch.zeros(1, device="cuda")
        s = call(torch.cuda.current_stream().cuda_stream)
    assert s == 5
    short = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    with pytest.raises(va.VerifyAttnError) as e:
        va.verify_attn_chunk(*held, b.scale, out=out, workspace=short)
    assert e.value.status == 5


@pytest.mark.parametrize("kind", KINDS)
def test_waits_that_run_out(kind):
    """A limit that no wait keeps: the call returns, says so, and the next one is right."""
    b = Chunk([40, 3], [700, 300], 8, 1, kind, 30)
    ws = torch.zeros(va.chunk_workspace_size(), dtype=torch.uint8, device="cuda")
    for given in (None, ws):
        va.last_device_error(given)
        va.set_wait_limit(1)
        try:
            for splits in (0, 1, 5):                   # (a wait that ends at once keeps any limit: a lone pair's do not)
                va.verify_attn_chunk(*b.args(), b.scale, k_descale=gpu(b.descales[0]), v_descale=gpu(b.descales[1]), k_scales=gpu(b.scales[0]),
                                     v_scales=gpu(b.scales[1]), workspace=given, num_splits=splits)
            torch.cuda.synchronize()
        finally:
            va.set_wait_limit(0)
        assert va.last_device_error(given) != 0 and va.last_device_error(given) == 0
        want, size = b.expect()
        assert (np.abs(decode(b.run(workspace=given)) - want) <= tolerance(b, want, size)).all()
        assert va.last_device_error(given) == 0
    check(b)


def test_softmax_of_the_verify_kernel():
    """The same batch through verify_attn: the two agree to their roundings."""
    b = Chunk([4, 3], [600, 900], 16, 1, "bf16", 31)
    a = b.args()
    x = va.verify_attn_chunk(*a, b.scale)
    y = va.verify_attn(*a, 4, 57 * 16, b.scale)
    torch.cuda.synchronize()
    want, size = b.expect()
    tol = tolerance(b, want, size)
    assert (np.abs(decode(x) - want) <= tol).all() and (np.abs(decode(x) - decode(y)) <= 2 * tol + 2.0 ** -7 * size).all()


@pytest.mark.parametrize("splits", [2, 3, 5, 7, 13, 31, 64, 75, 76, 1000])
def test_more_splits_than_units(splits):
    """Shares rounded up leave the last pairs nothing: they take part in nothing."""
    b = Chunk([2, 0, 1], [40, 9, 3], 2, 1, "bf16", 32)
    want, size = b.expect()
    assert (np.abs(decode(b.run(num_splits=splits)) - want) <= tolerance(b, want, size)).all()
    b = Chunk([70], [300], 8, 1, KINDS[1], 33)
    want, size = b.expect()
    assert (np.abs(decode(b.run(num_splits=splits)) - want) <= tolerance(b, want, size)).all()


def test_two_streams_at_once():
    """Calls that are under way together have workspaces of their own."""
    a, b = Chunk([300, 5], [4000, 900], 8, 1, "bf16", 34), Chunk([200], [5000], 16, 2, "scaled", 35)
    calls = []
    for x in (a, b):
        kw = dict(k_scales=gpu(x.scales[0]), v_scales=gpu(x.scales[1]))
        calls.append((x.args(), x.scale, kw, va.verify_attn_chunk(*x.args(), x.scale, **kw), torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (args, scale, kw, _, stream) in enumerate(calls):
            got[i].append(va.verify_attn_chunk(*args, scale, stream=stream, out=torch.empty_like(args[0]), **kw))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(calls[i][3], o) for o in got[i])
    assert va.last_device_error() == 0
