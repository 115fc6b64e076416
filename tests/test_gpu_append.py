"""append_kv and append_mla on the GPU against the fp64 oracle
(oracle/append_fp64.py): every cache kind, both rotations, ragged and empty
sequences, odd head counts, strides, page scales that grow, stay or hold
garbage, tokens without a place."""
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import Batch, check_kv, check_mla, gpu, raw, run_kv, run_mla

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "scaled"]
LENS = [([4, 2], [1024, 769]),
        ([1], [1]),
        ([1, 1, 1, 1], [16, 17, 31, 33]),
        ([3, 0, 4, 1, 2], [20, 5, 18, 0, 2]),       # no new token, S < L, straddled pages
        ([0, 0, 5, 0], [3, 0, 40, 16]),
        ([37, 16, 1, 130, 15], [37, 48, 300, 141, 31])]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("li", range(len(LENS)))
def test_append_kv(kind, interleaved, li):
    q, kv = LENS[li]
    hq, hkv, rot = [(16, 1, 256), (5, 1, 64), (12, 3, 128), (8, 2, 256), (1, 1, 8), (32, 2, 192)][li]
    check_kv(Batch(q, kv, hq, hkv, kind, rot, 100 * li + KINDS.index(kind), tail=li % 3, interleaved=interleaved))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rot", [0, 8, 16, 24, 40, 104, 248, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_partial_rotations(kind, rot, interleaved):
    check_kv(Batch([5, 20], [9, 41], 3, 2, kind, rot, 7 + rot, interleaved=interleaved))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("li", range(len(LENS)))
def test_append_mla(kind, interleaved, li):
    q, kv = LENS[li]
    hq = [16, 1, 3, 17, 64, 128][li]
    rot = 0 if li == 4 else 64
    check_mla(Batch(q, kv, hq, 1, kind, rot, 300 + 10 * li + KINDS.index(kind), dim=576, tail=li % 2,
                    interleaved=interleaved), fused=li % 2 == 0)


@pytest.mark.parametrize("mla", [False, True])
@pytest.mark.parametrize("old", [2.0 ** -30, 2.0 ** -9, 0.3, 2.0 ** 40, 0.0, -1.0, float("nan"), float("inf"), 1e-45])
def test_scales_of_pages_with_older_tokens(mla, old):
    b = Batch([1, 3, 2], [6, 20, 40], 4, 1 if mla else 2, "scaled", 64, 11, dim=576 if mla else 256)
    for s in b.scales:
        s.fill_(old)
    (check_mla if mla else check_kv)(b)


@pytest.mark.parametrize("mla", [False, True])
def test_scales_of_fresh_pages_ignore_what_was_there(mla):
    b = Batch([16, 33], [16, 65], 4, 1, "scaled", 64, 12, dim=576 if mla else 256)
    for c, s in zip(b.caches, b.scales):
        s.fill_(float("nan"))
        c.view(torch.uint8).fill_(0x7F)
    b.used[1], b.cu[2] = 64, 48                       # 32 tokens on a page boundary
    (check_mla if mla else check_kv)(b)


@pytest.mark.parametrize("size", [0.0, 448.0, 449.0, 3e38, 1e-39, 2.0 ** 73, 1.75 * 2.0 ** -56])
def test_scale_borders(size):
    """Zeros, the largest code exactly, one step above it, values at the ends of the exponent range."""
    b = Batch([2, 1], [2, 17], 1, 1, "scaled", 0, 13)
    for x in (b.k, b.v):
        x.zero_()
        x[:, 0, 5] = size
    b.k[:, 0, 9] = -size
    check_kv(b)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("mla", [False, True])
def test_infinities_and_nan_in_new_tokens(kind, mla):
    b = Batch([3, 2], [10, 34], 2, 1, kind, 0, 14, dim=576 if mla else 256)
    b.k[0, 0, 3], b.k[1, 0, 8], b.k[2, 0, -1] = float("nan"), float("-inf"), float("inf")
    b.v[3, 0, 0] = float("nan")
    b.v[4] = float("nan")
    (check_mla if mla else check_kv)(b)


@pytest.mark.parametrize("mla", [False, True])
@pytest.mark.parametrize("cu,used", [([0, 30, 10, 40, 24], [40, 30, 35, 20]), ([0, -5, 300, 24, 24], [40, 30, 35, 20]),
                                     ([0, 8, 8, 20, 2000000000], [-3, 2000000000, 0, 17])])
def test_broken_prefix_sums_stay_inside(mla, cu, used):
    """Prefix sums that decrease, are negative or pass the rows, and lengths that
    make no sense: unspecified rows, but nothing outside the tensors."""
    b = Batch([6, 6, 6, 6], [40, 30, 35, 20], 4, 1, "scaled", 64, 33, dim=576 if mla else 256)
    b.cu, b.used = torch.tensor(cu, dtype=torch.int32), torch.tensor(used, dtype=torch.int32)
    T, guard = b.q.shape[0], 4096
    wide = torch.full((T * 4 * 576 + 2 * guard,), 7.0, dtype=torch.bfloat16, device="cuda")
    cache = [torch.full((b.pages * 16 * 576 + 2 * guard,), 0x11, dtype=torch.uint8, device="cuda") for _ in range(2)]
    inner = [c[guard:guard + b.pages * 16 * b.dim].view(torch.float8_e4m3fn).view(b.pages, 16, 1, b.dim) for c in cache]
    scales = [torch.ones(b.pages, 1, device="cuda") for _ in range(2)]
    w = b.q.shape[2]
    q_out = wide[guard:guard + T * 4 * w].view(T, 4, w)
    if mla:
        row = gpu(b.k)[:, 0]
        va.append_mla(row[:, :512], row[:, 512:], inner[0], gpu(b.block_table), gpu(b.cu), gpu(b.used), q_pe=gpu(b.q), q_pe_out=q_out,
                      cos_sin=gpu(b.cos_sin), scales=scales[0])
    else:
        va.append_kv(gpu(b.k), gpu(b.v), *inner, gpu(b.block_table), gpu(b.cu), gpu(b.used), q=gpu(b.q), q_out=q_out,
                     cos_sin=gpu(b.cos_sin), k_scales=scales[0], v_scales=scales[1])
    torch.cuda.synchronize()
    assert (wide[:guard] == 7.0).all() and (wide[guard + T * 4 * w:] == 7.0).all()
    for c in cache:
        assert (c[:guard] == 0x11).all() and (c[guard + b.pages * 16 * b.dim:] == 0x11).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("mla", [False, True])
def test_pages_that_do_not_exist(kind, mla):
    """Bad page ids and positions past the table store nothing; q is still rotated."""
    b = Batch([4, 3, 20], [40, 35, 60], 4, 1 if mla else 2, kind, 64, 15, dim=576 if mla else 256)
    b.block_table[0, 2] = -1
    b.block_table[1, 2] = b.pages
    b.block_table = b.block_table[:, :3].contiguous()          # the third sequence's last page is outside
    (check_mla if mla else check_kv)(b)


@pytest.mark.parametrize("mla", [False, True])
def test_positions(mla):
    b = Batch([4, 3], [40, 35], 4, 1, "bf16", 64, 16, dim=576 if mla else 256)
    b.positions = torch.tensor([0, 39, 7, 100000, -5, 2, 2], dtype=torch.int32)
    (check_mla if mla else check_kv)(b)


@pytest.mark.parametrize("kind", KINDS)
def test_rotation_in_place(kind):
    b = Batch([4, 0, 3], [40, 7, 2], 6, 2, kind, 128, 17, tail=2)
    check_kv(b, in_place=True)


@pytest.mark.parametrize("kind", KINDS)
def test_strided_tensors(kind):
    """q, k, v as views of one projection; K and V pages interleaved in one
    tensor; scales interleaved; a transposed block table."""
    b = Batch([4, 2, 17], [40, 18, 33], 6, 2, kind, 64, 18)
    T = b.k.shape[0]
    ref = run_kv(b)
    qkv = torch.cat([b.q, b.k, b.v], dim=1).reshape(T, -1).to("cuda").reshape(T, 10, 256)
    both = torch.stack([gpu(b.caches[0]).view(torch.uint8), gpu(b.caches[1]).view(torch.uint8)], dim=1).view(b.caches[0].dtype)
    sc = None if b.scales[0] is None else torch.stack([gpu(s) for s in b.scales], dim=-1)
    q_out = torch.full((T, 6, 320), 7.0, dtype=torch.bfloat16, device="cuda")[..., 64:]
    btt = gpu(b.block_table).t().contiguous().t()
    va.append_kv(qkv[:, 6:8], qkv[:, 8:], both[:, 0], both[:, 1], btt, gpu(b.cu), gpu(b.used), q=qkv[:, :6], q_out=q_out,
                 cos_sin=gpu(b.cos_sin), k_descale=gpu(b.descales[0]), v_descale=gpu(b.descales[1]),
                 k_scales=None if sc is None else sc[..., 0], v_scales=None if sc is None else sc[..., 1])
    assert torch.equal(q_out, ref[1])
    for i in range(2):
        assert (raw(both[:, i]) == raw(ref[2][i])).all()
        if sc is not None:
            assert torch.equal(sc[..., i], ref[3][i])


@pytest.mark.parametrize("mla", [False, True])
def test_bf16_caches_take_descales(mla):
    b = Batch([4, 3], [40, 35], 4, 1, "bf16", 64, 31, dim=576 if mla else 256)
    b.descales = [torch.tensor([0.3]), torch.tensor([4.0])]
    (check_mla if mla else check_kv)(b)


@pytest.mark.parametrize("mla", [False, True])
def test_empty_batches(mla):
    run = run_mla if mla else run_kv
    b = Batch([], [], 2, 1, "bf16", 64, 19, dim=576 if mla else 256)
    out = run(b)
    caches = [out[2]] if mla else out[2]
    assert all((raw(c) == raw(w)).all() for c, w in zip(caches, b.caches))
    (check_mla if mla else check_kv)(Batch([0, 0], [5, 0], 2, 1, "scaled", 64, 20, dim=576 if mla else 256))


def test_many_sequences():
    """More sequences than a CTA has threads."""
    g = torch.Generator().manual_seed(3)
    q = torch.randint(0, 4, (700,), generator=g).tolist()
    kv = [n + int(x) for n, x in zip(q, torch.randint(0, 40, (700,), generator=g))]
    check_kv(Batch(q, kv, 2, 1, "scaled", 16, 21))
    check_mla(Batch(q[:600], kv[:600], 2, 1, "bf16", 64, 22, dim=576))


@pytest.mark.parametrize("kind", ["e4m3", "scaled"])
def test_offsets_past_32_bits(kind):
    """A cache of more than 2^31 elements: the last pages."""
    b = Batch([4, 3], [40, 35], 2, 1, kind, 64, 23)
    pages = (1 << 31) // (16 * 256) + 64
    big = [torch.zeros(pages, 16, 1, 256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    sc = [None, None] if kind != "scaled" else [torch.ones(pages, 1, device="cuda") for _ in range(2)]
    ref_c, ref_s = check_kv(b)
    at = pages - b.pages
    for i in range(2):
        big[i][at:] = gpu(b.caches[i]).view(torch.uint8).view(torch.float8_e4m3fn)
        if sc[i] is not None:
            sc[i][at:] = gpu(b.scales[i])
    va.append_kv(gpu(b.k), gpu(b.v), big[0], big[1], gpu(b.block_table) + at, gpu(b.cu), gpu(b.used), cos_sin=gpu(b.cos_sin),
                 k_descale=gpu(b.descales[0]), v_descale=gpu(b.descales[1]), k_scales=sc[0], v_scales=sc[1])
    for i in range(2):
        assert (raw(big[i][at:]) == raw(ref_c[i])).all()
        assert not big[i][:at].view(torch.uint8).any()
        if sc[i] is not None:
            assert torch.equal(sc[i][at:], ref_s[i])


def test_repeating_a_call_changes_nothing():
    """The same tokens again (a redrafted step): bytes and scales stay, and so
    do they after a longer draft was taken back."""
    b = Batch([4, 4], [21, 40], 2, 1, "scaled", 64, 24)
    caches, scales = check_kv(b)
    c2, s2 = [c.clone() for c in caches], [s.clone() for s in scales]
    va.append_kv(gpu(b.k), gpu(b.v), c2[0], c2[1], gpu(b.block_table), gpu(b.cu), gpu(b.used), cos_sin=gpu(b.cos_sin),
                 k_scales=s2[0], v_scales=s2[1])
    for i in range(2):
        assert (raw(c2[i]) == raw(caches[i])).all() and torch.equal(s2[i], scales[i])


@pytest.mark.parametrize("mla", [False, True])
def test_capture_and_replay(mla):
    """A captured call replayed on other tokens, lengths and pages equals the eager call."""
    a = Batch([4, 2, 3], [40, 18, 33], 4, 1, "scaled", 64, 25, dim=576 if mla else 256)
    b = Batch([3, 4, 2], [24, 33, 17], 4, 1, "scaled", 64, 26, dim=576 if mla else 256)
    b.block_table = torch.randperm(a.pages, generator=torch.Generator().manual_seed(1))[:9].reshape(3, 3).to(torch.int32)
    b.cos_sin = a.cos_sin
    st = {n: gpu(getattr(a, n)) for n in ("q", "k", "v", "block_table", "cu", "used", "cos_sin")}
    caches, scales = [gpu(c) for c in a.caches], [gpu(s) for s in a.scales]
    q_out = torch.zeros_like(st["q"])

    def call(x, caches, scales, q_out):
        if mla:
            va.append_mla(x["k"][:, 0, :512], x["k"][:, 0, 512:], caches[0], x["block_table"], x["cu"], x["used"], q_pe=x["q"],
                          q_pe_out=q_out, cos_sin=x["cos_sin"], scales=scales[0])
        else:
            va.append_kv(x["k"], x["v"], caches[0], caches[1], x["block_table"], x["cu"], x["used"], q=x["q"], q_out=q_out,
                         cos_sin=x["cos_sin"], k_scales=scales[0], v_scales=scales[1])

    call(st, caches, scales, q_out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(st, caches, scales, q_out)
    for n in st:
        st[n].copy_(getattr(b, n))
    for i in range(2):
        caches[i].view(torch.uint8).copy_(a.caches[i].view(torch.uint8))
        scales[i].copy_(a.scales[i])
    e_c, e_s, e_q = [gpu(c) for c in a.caches], [gpu(s) for s in a.scales], torch.zeros_like(q_out)
    call(st, e_c, e_s, e_q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, e_q)
    for i in range(1 if mla else 2):
        assert (raw(caches[i]) == raw(e_c[i])).all() and torch.equal(scales[i], e_s[i])


def test_side_stream_and_order():
    """On another stream than the current one, right behind the kernels that
    write its inputs there and before one that reads its outputs."""
    b = Batch([4, 2, 30], [40, 18, 33], 4, 1, "scaled", 64, 27)
    ref = run_kv(b)
    s = torch.cuda.Stream()
    for _ in range(5):
        caches, scales = [gpu(c) for c in b.caches], [gpu(x) for x in b.scales]
        k, v, q = torch.zeros_like(gpu(b.k)), torch.zeros_like(gpu(b.v)), gpu(b.q)
        kk, vv = gpu(b.k), gpu(b.v)
        bt, cu, used, cs = gpu(b.block_table), gpu(b.cu), gpu(b.used), gpu(b.cos_sin)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            k.copy_(kk)
            v.copy_(vv)
        q_out = torch.zeros_like(q)
        s.wait_stream(torch.cuda.current_stream())
        va.append_kv(k, v, caches[0], caches[1], bt, cu, used, q=q, q_out=q_out, cos_sin=cs, k_scales=scales[0],
                     v_scales=scales[1], stream=s)
        with torch.cuda.stream(s):
            got = [c.clone() for c in caches]
            k.zero_()
        torch.cuda.synchronize()
        assert torch.equal(q_out, ref[1])
        assert all((raw(a) == raw(c)).all() for a, c in zip(got, ref[2]))


@pytest.mark.parametrize("kind", KINDS)
def test_long_prompt(kind):
    """A prompt of thousands of tokens, every byte against the same formula in torch."""
    T = 5003
    b = Batch([T, 1], [T + 37, 9], 2, 1, kind, 256, 28)
    _, q_out, caches, scales = run_kv(b)
    cs = b.cos_sin[37:37 + T]
    cos, sin = cs[:, None, :128], cs[:, None, 128:]
    k = b.k[:T].float()
    y = torch.cat([k[..., :128] * cos - k[..., 128:] * sin, k[..., 128:] * cos + k[..., :128] * sin], dim=-1)
    pos = torch.arange(37, 37 + T)
    page, slot = b.block_table[0, pos // 16].long(), pos % 16
    got = raw(caches[0])[page.numpy(), slot.numpy()]
    if kind == "bf16":
        want = y.to(torch.bfloat16)
    elif kind == "e4m3":
        want = (y / b.descales[0]).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        want = (y / scales[0].cpu()[page][:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert (got == raw(want)).all()
