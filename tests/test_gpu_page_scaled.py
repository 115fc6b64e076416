"""Verify attention over page-scaled e4m3 caches on the GPU against the fp64
oracle (oracle/page_scaled_fp64.py): element by element within the bound of the
kernels' roundings, and by the relative L2 gates of the other paths."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import decode, descriptors
from oracle.page_scaled_fp64 import page_scaled_oracle
from parity_gate import check_gates
from speculative_decoding_verify_split_gb300.workloads import make_mla_workload, make_workload

pytestmark = pytest.mark.gpu


def scales_for(w, seed, spread=6.0, powers=True):
    """Scales of every page and head, a factor of 2^spread or so around 1."""
    cache = w.k_cache if hasattr(w, "k_cache") else w.kv_cache
    g = torch.Generator().manual_seed(seed)
    e = [(torch.rand(cache.shape[0], cache.shape[2], generator=g) - 0.5) * spread for _ in range(2)]
    if powers:
        e = [x.round() for x in e]
    ks, vs = torch.exp2(e[0]), torch.exp2(e[1])
    return ks / ks.max(), vs                     # K's at most 1: the logits stay those of a softmax in use


def finite(cache):
    return np.nan_to_num(decode(cache))          # NaN stands where nothing may be read


def oracle(w, ks, vs, **kw):
    k, v = finite(w.k_cache.cpu()), finite(w.v_cache.cpu())
    return page_scaled_oracle(decode(w.q.cpu()), k, v, ks.numpy(), vs.numpy(), w.block_table.cpu().numpy(),
                              w.cu_seqlens_q.cpu().numpy(), w.seqused_k.cpu().numpy(), w.softmax_scale, **kw)


def oracle_mla(w, s):
    c = finite(w.kv_cache.cpu())
    return page_scaled_oracle(decode(w.q.cpu()), c, c[..., :512], s.numpy(), s.numpy(), w.block_table.cpu().numpy(),
                              w.cu_seqlens_q.cpu().numpy(), w.seqused_k.cpu().numpy(), w.softmax_scale)


def compare(got, ref, tol, gates=True):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    bad = np.abs(g - ref) > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside the bound, worst {np.abs(g - ref)[bad].max()}"
    if gates:
        check_gates(g, ref)


def run(w, ks, vs, **kw):
    out = torch.full_like(w.q, float("nan"))
    va.verify_attn_scaled(w.q, w.k_cache, w.v_cache, ks.cuda(), vs.cuda(), w.block_table, w.cu_seqlens_q, w.seqused_k, w.max_seqlen_q,
                          w.max_seqlen_k, w.softmax_scale, out=out, **kw)
    torch.cuda.synchronize()
    return out


def run_mla(w, s, **kw):
    out = torch.full((*w.q.shape[:2], 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    va.verify_attn_mla_scaled(w.q, w.kv_cache, s.cuda(), w.block_table, w.cu_seqlens_q, w.seqused_k, w.max_seqlen_q, w.max_seqlen_k,
                              w.softmax_scale, out=out, **kw)
    torch.cuda.synchronize()
    return out


CASES = [dict(q=[4, 2, 3, 1, 4], kv=[1000, 769, 300, 5, 3], hq=16, hkv=1),
         dict(q=[2, 3, 4], kv=[2100, 513, 130], hq=32, hkv=2),
         dict(q=[1], kv=[1], hq=1, hkv=1),
         dict(q=[1, 1, 1, 1, 1, 1], kv=[15, 16, 17, 127, 128, 129], hq=20, hkv=4),
         dict(q=[3, 0, 2, 1, 4], kv=[700, 50, 0, 1, 2], hq=5, hkv=1),          # no draft token, no key, S < L
         dict(q=[2, 2], kv=[3000, 2500], hq=64, hkv=2)]


def workload(ci, seed):
    c = CASES[ci]
    return make_workload(c["q"], c["kv"], c["hq"], c["hkv"], "fp8_e4m3", seed=seed).to("cuda")


@pytest.mark.parametrize("ci", range(len(CASES)))
@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("splits", [0, 1, 7])
def test_scaled(ci, powers, splits):
    """All CTAs, one CTA (from 16 tiles on: Q in tensor memory), a few."""
    w = workload(ci, 500 + ci)
    ks, vs = scales_for(w, ci, powers=powers)
    compare(run(w, ks, vs, num_splits=splits), *oracle(w, ks, vs))


def test_both_layouts_are_covered():
    c = CASES[1]
    assert va.plan(3, 2, 32, 4, 2112, "fp8_e4m3", 152, 1)["kernel"] == 2
    assert va.plan(3, 2, 32, 4, 2112, "fp8_e4m3", 152, 0)["kernel"] == 1
    assert max(c["kv"]) <= 2112


@pytest.mark.parametrize("ci", range(len(CASES)))
@pytest.mark.parametrize("kw", [dict(window_left=0), dict(window_left=17), dict(window_left=300), dict(softcap=3.0),
                                dict(window_left=100, softcap=20.0, sinks=True), dict(sinks=True)])
def test_variants(ci, kw):
    w = workload(ci, 520 + ci)
    ks, vs = scales_for(w, 40 + ci)
    kw = dict(kw)
    okw = dict(kw)
    if kw.pop("sinks", None):
        kw["sinks"] = torch.linspace(-3, 3, w.q.shape[1], device="cuda")
        okw["sinks"] = kw["sinks"].cpu().numpy().astype(np.float64)
    ref = oracle(w, ks, vs, **okw)
    for splits in (0, 2):
        compare(run(w, ks, vs, num_splits=splits, **kw), *ref)


@pytest.mark.parametrize("hq", [1, 3, 8, 16])
@pytest.mark.parametrize("splits", [0, 1, 5])
def test_latent(hq, splits):
    q, kv = [4, 2, 3, 1, 2, 0], [1000, 769, 130, 5, 1, 9]
    if hq == 1:
        q, kv = [1, 1], [1, 3000]
    w = make_mla_workload(q, kv, hq, "fp8_e4m3", seed=540 + hq).to("cuda")
    s, _ = scales_for(w, hq, spread=4.0)
    compare(run_mla(w, s, num_splits=splits), *oracle_mla(w, s))


@pytest.mark.parametrize("hq,q", [(1, 1), (15, 1), (16, 1), (17, 1), (16, 2), (8, 4), (11, 3), (16, 3), (49, 1), (16, 4)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_latent_rows_and_rising_scales(hq, q, splits):
    """Packed rows around 16, 32 and 48 (the sizes at which the latent kernel
    lays P and its accumulator out differently), over pages whose scales rise
    along the sequence, so that the reference of a row moves again and again."""
    w = make_mla_workload([q, q, max(1, q - 1)], [2500, 700, 70], hq, "fp8_e4m3", seed=560 + hq + q).to("cuda")
    s = torch.ones(w.kv_cache.shape[0], 1)
    table = w.block_table.cpu()
    for b, n in enumerate(w.seqused_k.tolist()):
        pages = -(-n // 16)
        s[table[b, :pages].long(), 0] = torch.exp2((torch.arange(pages) * 10 // pages - 9).float() / 2)
    compare(run_mla(w, s, num_splits=splits), *oracle_mla(w, s))


@pytest.mark.parametrize("mla", [False, True])
def test_scales_far_apart(mla):
    """V's scales from 2^-40 to 2^40 over the pages, and K's so that the keys
    of the small ones carry the row: the weights are still right."""
    if mla:
        w = make_mla_workload([2, 1], [600, 300], 16, "fp8_e4m3", seed=550).to("cuda")
        s = torch.exp2(torch.arange(w.kv_cache.shape[0]).float() % 21 - 20)[:, None]     # keys and values share it
        compare(run_mla(w, s), *oracle_mla(w, s), gates=False)
        return
    w = make_workload([2, 1], [600, 300], 16, 1, "fp8_e4m3", seed=551).to("cuda")
    n = w.k_cache.shape[0]
    e = (torch.arange(n).float() * 37) % 81 - 40
    ks, vs = torch.exp2(-e / 20 - 2)[:, None], torch.exp2(e)[:, None]
    compare(run(w, ks, vs), *oracle(w, ks, vs), gates=False)


@pytest.mark.parametrize("value", [0.0, -2.0, float("nan"), float("inf"), 1e-30, 3.4e38])
def test_scales_outside_their_range(value):
    """A page with such a V scale is read by the clamped one; beside it the others."""
    w = make_workload([2, 1], [90, 300], 8, 1, "fp8_e4m3", seed=552).to("cuda")
    ks, vs = scales_for(w, 3)
    vs[int(w.block_table[0, 1])] = value
    if not value > 1:                            # a K scale of 2^64 leaves no softmax to compare
        ks[int(w.block_table[1, 2])] = value
    compare(run(w, ks, vs), *oracle(w, ks, vs), gates=False)


def test_pages_nobody_sees_may_hold_anything():
    """NaN scales on pages past the lengths, on unused pages and, with a
    window, before it (ids that do not exist there)."""
    w = make_workload([2, 3], [300, 513], 8, 2, "fp8_e4m3", seed=553).to("cuda")
    ks, vs = scales_for(w, 4)
    ref = oracle(w, ks, vs, window_left=60)
    used = set()
    bt = w.block_table.clone()
    for b, (L, S) in enumerate(((2, 300), (3, 513))):
        first = max(0, S - L - 60) // 16
        used |= set(bt[b, first:-(-S // 16)].tolist())
        bt[b, :first] = torch.where(torch.arange(first, device="cuda") % 2 == 0, -7, w.k_cache.shape[0] + 5).to(torch.int32)
    for i in range(ks.shape[0]):
        if i not in used:
            ks[i] = vs[i] = float("nan")
    w.block_table = bt
    compare(run(w, ks, vs, window_left=60), *ref)


def test_interleaved_scales_and_strided_tensors():
    w = make_workload([2, 3], [300, 513], 8, 2, "fp8_e4m3", seed=554).to("cuda")
    ks, vs = scales_for(w, 5)
    ref = run(w, ks, vs)
    both = torch.stack([ks, vs], dim=-1).cuda()
    wide = torch.zeros(w.q.shape[0], 8, 512, dtype=torch.bfloat16, device="cuda")
    out = torch.full((w.q.shape[0], 8, 320), float("nan"), dtype=torch.bfloat16, device="cuda")[..., 64:]
    q = wide[..., 256:]
    q.copy_(w.q)
    kv = torch.stack([w.k_cache.view(torch.uint8), w.v_cache.view(torch.uint8)], dim=1).view(w.k_cache.dtype)
    va.verify_attn_scaled(q, kv[:, 0], kv[:, 1], both[..., 0], both[..., 1], w.block_table.t().contiguous().t(), w.cu_seqlens_q,
                          w.seqused_k, w.max_seqlen_q, w.max_seqlen_k, w.softmax_scale, out=out)
    assert torch.equal(out, ref)


def test_equal_scales_give_the_descaled_call():
    """One power of two everywhere: the bits of verify_attn with that descale,
    for the same split of the keys (which alone decides the order of sums)."""
    w = make_workload([4, 2], [1024, 769], 16, 1, "fp8_e4m3", seed=555, k_descale=0.5, v_descale=1.0).to("cuda")
    n = w.k_cache.shape[0]
    m = make_mla_workload([4, 2], [1024, 769], 16, "fp8_e4m3", seed=556).to("cuda")
    for splits in (1, 7, 16):
        got = run(w, torch.full((n, 1), 0.5), torch.ones(n, 1), num_splits=splits)
        assert torch.equal(got, va.run_workload_ex(w, num_splits=splits))
        got = run_mla(m, torch.ones(m.kv_cache.shape[0], 1), num_splits=splits)
        assert torch.equal(got, va.run_mla_workload(m, num_splits=splits))


def test_empty_batches():
    w = make_workload([0, 0], [5, 0], 4, 1, "fp8_e4m3", seed=557).to("cuda")
    with pytest.raises(va.VerifyAttnError) as e:      # a bound of 0 draft tokens is refused, as by verify_attn
        run(w, *scales_for(w, 1))
    assert w.max_seqlen_q == 0 and e.value.status == 4
    w.max_seqlen_q = 1
    assert run(w, *scales_for(w, 1)).shape[0] == 0
    w = make_workload([2, 2], [0, 0], 4, 1, "fp8_e4m3", seed=558).to("cuda")
    assert not run(w, *scales_for(w, 1)).any()


def test_rows_behind_the_last_sequence_stay():
    w = make_workload([2, 3], [300, 513], 8, 2, "fp8_e4m3", seed=559).to("cuda")
    ks, vs = scales_for(w, 5)
    ref = run(w, ks, vs)
    w.q = torch.cat([w.q, torch.ones_like(w.q[:2])])
    out = torch.full_like(w.q, 5.0)
    va.verify_attn_scaled(w.q, w.k_cache, w.v_cache, ks.cuda(), vs.cuda(), w.block_table, w.cu_seqlens_q, w.seqused_k, w.max_seqlen_q,
                          w.max_seqlen_k, w.softmax_scale, out=out)
    assert torch.equal(out[:5], ref) and (out[5:] == 5.0).all()


def test_page_and_scale_offsets_past_32_bits():
    """The last pages of a cache of more than 2^31 elements, scales 2^12 apart."""
    w = make_workload([2, 3], [40, 513], 8, 1, "fp8_e4m3", seed=560).to("cuda")
    ks, vs = scales_for(w, 6)
    ref = run(w, ks, vs)
    n = w.k_cache.shape[0]
    pages = (1 << 31) // 4096 + 64
    at = pages - n
    big = [torch.full((pages, 16, 1, 256), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    sc = [torch.full((pages, 4104), float("nan"), device="cuda")[:, 4096:4097] for _ in range(2)]
    for dst, src in zip(big + sc, (w.k_cache, w.v_cache, ks.cuda(), vs.cuda())):
        if src.dtype == torch.float8_e4m3fn:
            dst[at:].view(torch.uint8).copy_(src.view(torch.uint8))
        else:
            dst[at:].copy_(src)
    got = va.verify_attn_scaled(w.q, big[0], big[1], sc[0], sc[1], w.block_table + at, w.cu_seqlens_q, w.seqused_k, w.max_seqlen_q,
                                w.max_seqlen_k, w.softmax_scale)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("mla", [False, True])
def test_two_streams_and_two_graphs(mla):
    """Calls without a workspace at the same time on two streams, and two
    captured ones replayed together: none shares memory with another."""
    ws, ss, refs = [], [], []
    for i in range(2):
        w = (make_mla_workload([4, 2, 1], [3000, 900, 77], 16, "fp8_e4m3", seed=570 + i) if mla else
             make_workload([4, 2, 1], [3000, 900, 77], 16, 1, "fp8_e4m3", seed=570 + i)).to("cuda")
        s = [x.cuda() for x in scales_for(w, i)]
        ws.append(w)
        ss.append(s)
        refs.append(run_mla(w, s[0]) if mla else run(w, *s))

    def call(i, out):
        w = ws[i]
        if mla:
            va.verify_attn_mla_scaled(w.q, w.kv_cache, ss[i][0], w.block_table, w.cu_seqlens_q, w.seqused_k, w.max_seqlen_q,
                                      w.max_seqlen_k, w.softmax_scale, out=out)
        else:
            va.verify_attn_scaled(w.q, w.k_cache, w.v_cache, *ss[i], w.block_table, w.cu_seqlens_q, w.seqused_k, w.max_seqlen_q,
                                  w.max_seqlen_k, w.softmax_scale, out=out)

    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(refs[i]) for _ in range(20)] for i in range(2)]
    torch.cuda.synchronize()
    for k in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                call(i, outs[i][k])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, refs[i]) for o in outs[i])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            call(i, outs[i][0])
        outs[i][0].zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], refs[i])


def test_capture_without_a_workspace_is_refused_by_the_library():
    """The C call's own workspace may be replaced later: not during capture."""
    w = make_workload([2], [40], 4, 1, "fp8_e4m3", seed=580).to("cuda")
    m = make_mla_workload([2], [40], 4, "fp8_e4m3", seed=581).to("cuda")
    ks, vs = [x.cuda() for x in scales_for(w, 1)]
    ms = torch.ones(m.kv_cache.shape[0], 1, device="cuda")
    out, mout = torch.zeros_like(w.q), torch.zeros(2, 4, 512, dtype=torch.bfloat16, device="cuda")
    codes = []

    def calls(stream):
        r = descriptors(w.q, w.k_cache, w.v_cache, ks, vs, w.block_table, w.cu_seqlens_q, w.seqused_k, out)
        codes.append(va.library().verify_attn_scaled(*r[:8], 2, w.max_seqlen_k, 0.1, r[8], None, None, 0, 0, None, stream))
        r = descriptors(m.q, m.kv_cache, ms, m.block_table, m.cu_seqlens_q, m.seqused_k, mout)
        codes.append(va.library().verify_attn_mla_scaled(*r[:6], 2, m.max_seqlen_k, 0.1, r[6], None, 0, 0, None, stream))

    calls(torch.cuda.current_stream().cuda_stream)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls(torch.cuda.current_stream().cuda_stream)
        out.fill_(1.0)
    assert codes == [0, 0, 5, 5]


@pytest.mark.parametrize("mla", [False, True])
def test_waits_that_run_out(mla):
    """With a limit of 1 ns the call returns with a status; the next one is right."""
    if mla:
        w = make_mla_workload([4, 2, 3], [2500, 700, 130], 16, "fp8_e4m3", seed=590).to("cuda")
        n = va.mla_workspace_size(w.q, w.seqused_k, w.max_seqlen_q, w.max_seqlen_k)
    else:
        w = make_workload([4, 2, 3], [2500, 700, 130], 16, 1, "fp8_e4m3", seed=591).to("cuda")
        n = va.workspace_size(w.q, w.k_cache, w.seqused_k, w.max_seqlen_q, w.max_seqlen_k)
    ws = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    ks, vs = scales_for(w, 7)
    call = (lambda **kw: run_mla(w, ks, workspace=ws, **kw)) if mla else (lambda **kw: run(w, ks, vs, workspace=ws, **kw))
    va.set_wait_limit(1)
    try:
        for splits in (0, 1, 5):
            call(num_splits=splits)
        if not mla:
            call(window_left=300, softcap=20.0)
    finally:
        va.set_wait_limit(0)
    assert va.last_device_error(ws) != 0 and va.last_device_error(ws) == 0
    for splits in (0, 1):
        compare(call(num_splits=splits), *(oracle_mla(w, ks) if mla else oracle(w, ks, vs)))
    assert va.last_device_error(ws) == 0


@pytest.mark.parametrize("hq,q,kv", [(16, [4, 2], [1024, 769]), (16, [1, 1], [500, 40]), (8, [3], [100]), (12, [1, 4, 2], [30, 17, 700]),
                                     (64, [1], [2000])])
def test_small_batches_in_the_promised_workspace(hq, q, kv):
    """Small batches run as clusters: in exactly the workspace that the size call
    names, with garbage in it."""
    w = make_workload(q, kv, hq, 1, "fp8_e4m3", seed=595).to("cuda")
    ks, vs = scales_for(w, 8)
    n = va.workspace_size(w.q, w.k_cache, w.seqused_k, w.max_seqlen_q, w.max_seqlen_k)
    ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:n]
    compare(run(w, ks, vs, workspace=ws), *oracle(w, ks, vs))
    m = make_mla_workload(q, kv, hq, "fp8_e4m3", seed=596).to("cuda")
    s, _ = scales_for(m, 9, spread=4.0)
    n = va.mla_workspace_size(m.q, m.seqused_k, m.max_seqlen_q, m.max_seqlen_k)
    ws = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    ws = ws[(-ws.data_ptr()) % 256:][:n]
    compare(run_mla(m, s, workspace=ws), *oracle_mla(m, s))


# (sequences, KV heads, query heads, tokens, keys): clusters of 8, 4, 2 and 1
# CTAs, with a KV head's query heads in one to sixteen of them, more sequences
# than the kernels cache, and batches just past the clusters' reach
CLUSTERS = [(1, 1, 16, [1], [900]), (1, 1, 64, [1], [130]), (2, 2, 32, [4], [700, 40]), (5, 1, 16, [4, 1], [1000, 300, 17]),
            (7, 2, 6, [3], [500, 1]), (16, 1, 16, [2], [600, 513, 128]), (20, 1, 8, [4], [400, 129]), (33, 1, 5, [1, 0, 2], [300, 0, 64]),
            (38, 2, 8, [2], [200, 127]), (70, 1, 4, [1], [150, 90, 1]), (76, 2, 4, [3], [100, 33]), (80, 2, 8, [1], [260, 16]),
            (153, 1, 16, [1], [100, 20]), (600, 1, 2, [1, 2, 0], [40, 5, 17])]


@pytest.mark.parametrize("ci", range(len(CLUSTERS)))
@pytest.mark.parametrize("kw", [{}, dict(window_left=50, softcap=10.0, sinks=True)])
def test_batches_of_every_size(ci, kw):
    B, hkv, hq, q, kv = CLUSTERS[ci]
    q, kv = [q[i % len(q)] for i in range(B)], [kv[i % len(kv)] for i in range(B)]
    w = make_workload(q, kv, hq, hkv, "fp8_e4m3", seed=620 + ci).to("cuda")
    ks, vs = scales_for(w, 60 + ci)
    kw, okw = dict(kw), dict(kw)
    if kw.get("sinks"):
        kw["sinks"] = torch.linspace(-3, 3, hq, device="cuda")
        okw["sinks"] = kw["sinks"].cpu().numpy().astype(np.float64)
    compare(run(w, ks, vs, **kw), *oracle(w, ks, vs, **okw))
    if hkv == 1 and not kw:
        m = make_mla_workload(q, kv, hq, "fp8_e4m3", seed=640 + ci).to("cuda")
        s, _ = scales_for(m, 80 + ci, spread=4.0)
        compare(run_mla(m, s), *oracle_mla(m, s))


@pytest.mark.parametrize("scale", [-0.0625, 0.0, 0.2])
def test_sign_of_the_softmax_scale(scale):
    w = make_workload([4, 2], [300, 130], 16, 1, "fp8_e4m3", seed=660).to("cuda")
    m = make_mla_workload([4, 2], [300, 130], 16, "fp8_e4m3", seed=661).to("cuda")
    w.softmax_scale, m.softmax_scale = scale, scale / 3
    ks, vs = scales_for(w, 9)
    s, _ = scales_for(m, 10, spread=4.0)
    for splits in (0, 1, 3):
        compare(run(w, ks, vs, num_splits=splits), *oracle(w, ks, vs))
        compare(run_mla(m, s, num_splits=splits), *oracle_mla(m, s))


def test_back_to_back_calls_on_changing_inputs():
    """Unsynchronised calls whose inputs kernels rewrite right before each: the
    results of the calls made alone (clusters, and the split over all CTAs)."""
    for splits in (0, 5):
        ws = [make_workload([4, 2, 3], [500, 129, 64], 16, 1, "fp8_e4m3", seed=670 + i).to("cuda") for i in range(2)]
        sc = [[x.cuda() for x in scales_for(w, i)] for i, w in enumerate(ws)]
        ref = [run(w, *s, num_splits=splits) for w, s in zip(ws, sc)]
        cur, cs = ws[0], [x.clone() for x in sc[0]]
        bufs = [cur.q.clone(), cur.k_cache.clone(), cur.v_cache.clone(), cur.block_table.clone()]
        outs = []
        for k in range(12):
            w, s = ws[k % 2], sc[k % 2]
            for dst, src in zip(bufs + cs, [w.q, w.k_cache, w.v_cache, w.block_table] + s):
                (dst.view(torch.uint8) if dst.dtype == torch.float8_e4m3fn else dst).copy_(
                    src.view(torch.uint8) if src.dtype == torch.float8_e4m3fn else src)
            outs.append(va.verify_attn_scaled(*bufs[:3], *cs, bufs[3], w.cu_seqlens_q, w.seqused_k, w.max_seqlen_q, w.max_seqlen_k,
                                              w.softmax_scale, num_splits=splits))
        torch.cuda.synchronize()
        assert all(torch.equal(o, ref[k % 2]) for k, o in enumerate(outs))


def test_workspace_errors():
    w = make_workload([2], [2000], 4, 1, "fp8_e4m3", seed=592).to("cuda")
    ks, vs = scales_for(w, 7)
    with pytest.raises(va.VerifyAttnError) as e:
        run(w, ks, vs, workspace=torch.zeros(512, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 5


@pytest.mark.parametrize("scale", [-0.0625, 0.0, 0.2])
@pytest.mark.parametrize("hq,q", [(8, 1), (16, 1), (16, 4)])
def test_latent_sign_of_the_softmax_scale_and_size_of_q(scale, hq, q):
    """Both ways of staging Q (one row group and more), with heads from 2^-20
    times their size up (to 2^20 where the softmax scale is 0) and an all-zero
    row: each row has its own power of two."""
    w = make_mla_workload([q, q], [900, 200], hq, "fp8_e4m3", seed=570 + hq + q).to("cuda")
    s, _ = scales_for(w, hq, spread=2.0)
    e = torch.linspace(-20, 20 if scale == 0.0 else 0, hq, device="cuda").round()
    w.q.copy_((w.q.float() * torch.exp2(e)[None, :, None]).to(torch.bfloat16))
    w.q[0, 0] = 0
    w.softmax_scale = scale
    for splits in (0, 1):
        compare(run_mla(w, s, num_splits=splits), *oracle_mla(w, s), gates=False)
