"""The operators around a paged cache beyond the verify step: what each
computes, in plain torch, and the cases they are measured on.

Caches have 16-token pages, head_dim 256, and hold bf16, e4m3 with one descale
a tensor, or e4m3 with a power-of-two scale for each page and KV head.

* ``chunk``: causal attention of chunks of new tokens (whole prompts, pieces of
  prompts behind cached tokens, single tokens, mixed in a batch) over the paged
  cache, optionally with a sliding window beside which the first tokens of the
  sequence stay visible, a soft cap and per-head sinks in the normaliser.
* ``norm_append``: the new tokens' queries and keys are normalised head by head
  (root mean square over the head's 256 columns, times a learned weight),
  rotated by their positions, and keys and values stored in their pages.
* ``branch``: sequences of a page pool that share pages. A round of sampling:
  the rows of the last round's candidates are freed, each prompt is forked into
  new candidates (pages shared, counted in ``refs``), the candidates get room
  for their next tokens (a shared page that is about to be written is replaced
  by a page of their own), and the replaced pages' contents are copied.
* ``copy``: pages of K and V caches, with their scales, to other pages.

Token t of sequence b (L new tokens, S cached tokens with them) is at position
S - L + t. Free pages are those with refs 0; the k-th page that a call needs, in
the order of sequences and of places in their rows, is the k-th free one.
"""
import math
import random

import torch

own = False

PAGE = 16
DIM = 256
FP8 = torch.float8_e4m3fn


# ---- cases --------------------------------------------------------------------


def listed():
    return [
        # two short continuations of a chat behind a cached prefix: the latency of a small call
        dict(name="chunk_tiny_bf16", op="chunk", lens=1, seqs=2, q_lo=17, q_hi=48, kv_lo=200, kv_hi=1024, hq=16, hkv=1,
             cache="bf16", window=-1, first=0, softcap=0.0, sinks=False),
        # whole prompts of a small batch, nothing cached before them
        dict(name="chunk_prompts_bf16", op="chunk", lens=2, seqs=4, q_lo=700, q_hi=2500, kv_lo=1, kv_hi=1, hq=16, hkv=2,
             cache="bf16", window=-1, first=0, softcap=0.0, sinks=False),
        # pieces of prompts behind cached prefixes, page scales
        dict(name="chunk_prefix_scaled", op="chunk", lens=3, seqs=8, q_lo=256, q_hi=700, kv_lo=2000, kv_hi=16384, hq=16, hkv=1,
             cache="scaled", window=-1, first=0, softcap=0.0, sinks=False),
        # the last piece of a very long prompt
        dict(name="chunk_long_e4m3", op="chunk", lens=4, seqs=1, q_lo=2048, q_hi=2048, kv_lo=131072, kv_hi=131072, hq=16, hkv=1,
             cache="e4m3", window=-1, first=0, softcap=0.0, sinks=False),
        # single tokens of long streams: a window, four first tokens that stay visible, soft cap and sinks
        dict(name="chunk_single_first_tokens", op="chunk", lens=5, seqs=32, q_lo=1, q_hi=1, kv_lo=5000, kv_hi=32768, hq=32, hkv=2,
             cache="bf16", window=4095, first=4, softcap=30.0, sinks=True),
        # one verify step of two users of a model with query and key norms
        dict(name="norm_append_tiny_bf16", op="norm_append", lens=6, seqs=2, q_lo=2, q_hi=4, kv_lo=769, kv_hi=1024, hq=16, hkv=1,
             cache="bf16", rot=256, interleaved=False, offset=0.0, weights="bf16"),
        # a high-concurrency verify step, ragged draft counts, per-tensor descales, part of the head rotated
        dict(name="norm_append_many_e4m3", op="norm_append", lens=7, seqs=256, q_lo=1, q_hi=4, kv_lo=64, kv_hi=1024, hq=8, hkv=1,
             cache="e4m3", rot=128, interleaved=True, offset=1.0, weights="fp32"),
        # the prompts of a batch behind cached prefixes of odd length
        dict(name="norm_append_prompt_scaled", op="norm_append", lens=8, seqs=8, q_lo=513, q_hi=4096, kv_lo=700, kv_hi=5000, hq=32, hkv=2,
             cache="scaled", rot=256, interleaved=False, offset=0.0, weights="bf16"),
        # three candidates for each of four short prompts
        dict(name="branch_tiny", op="branch", lens=9, parents=4, children=3, kv_lo=100, kv_hi=1000, add=4, pool=1024, hkv=1, cache="bf16"),
        # seven candidates for each of 64 prompts
        dict(name="branch_many_scaled", op="branch", lens=10, parents=64, children=7, kv_lo=500, kv_hi=4096, add=20, pool=32768, hkv=1, cache="scaled"),
        # a few pages
        dict(name="copy_few_bf16", op="copy", pool=512, count=12, hkv=1, cache="bf16"),
        # prefixes to other pages of a cache with page scales
        dict(name="copy_many_scaled", op="copy", pool=24576, count=9001, hkv=2, cache="scaled"),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["chunk", "chunk", "chunk", "norm_append", "norm_append", "branch", "copy"])
    c = dict(op=op, lens=rng.randrange(1 << 30), hkv=rng.choice([1, 1, 2, 3, 4]), cache=rng.choice(["bf16", "e4m3", "scaled"]))
    if op == "copy":
        c["count"] = logint(1, 8192)
        c["pool"] = 2 * c["count"] + rng.randrange(1, 300)
        return c
    if op == "branch":
        c["hkv"] = rng.choice([1, 1, 2])
        c["parents"], c["children"] = logint(1, 64), rng.choice([1, 2, 3, 7])
        c["kv_hi"] = logint(20, 4096)
        c["kv_lo"] = max(1, c["kv_hi"] // rng.choice([1, 2, 20]))
        c["add"] = rng.choice([1, 4, 5, 16, 40])
        c["pool"] = c["parents"] * (-(-c["kv_hi"] // PAGE) + c["children"] * (c["add"] // PAGE + 2)) + rng.randrange(1, 500)
        return c
    if op == "norm_append":
        c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 5, 8])
        c["rot"] = rng.choice([32, 64, 128, 192, 256])
        c["interleaved"] = rng.random() < 0.5
        c["offset"] = rng.choice([0.0, 1.0])
        c["weights"] = rng.choice(["bf16", "fp32"])
        if rng.random() < 0.5:  # verify steps
            c.update(seqs=logint(1, 256), q_lo=rng.choice([0, 1, 2]), q_hi=rng.choice([2, 3, 4]), kv_lo=rng.choice([4, 17, 300]), kv_hi=logint(301, 4096))
        else:  # prompts
            c.update(seqs=rng.choice([1, 2, 3, 5, 8]), q_hi=logint(17, 2048))
            c["q_lo"] = max(1, c["q_hi"] // rng.choice([1, 2, 7]))
            c["kv_lo"] = c["q_hi"] + rng.choice([0, 1, 100])
            c["kv_hi"] = c["kv_lo"] + logint(1, 2048)
        return c
    c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 5, 8, 16])
    c["q_hi"] = logint(1, 2048)
    c["q_lo"] = max(1, c["q_hi"] // rng.choice([1, 2, 9]))
    c["kv_hi"] = logint(40, 65536)
    c["kv_lo"] = max(1, c["kv_hi"] // rng.choice([1, 2, 30]))
    # the plain form holds the logits of the padded batch
    c["seqs"] = max(1, min(logint(1, 64), int(1.0e9 // (c["hq"] * c["q_hi"] * max(c["q_hi"], c["kv_hi"])))))
    variants = rng.random() < 0.4
    c["window"] = rng.choice([-1, 0, 63, 500, 4000]) if variants else -1
    c["first"] = rng.choice([0, 1, 4, 130]) if variants and c["window"] >= 0 else 0
    c["softcap"] = rng.choice([0.0, 15.0, 30.0]) if variants else 0.0
    c["sinks"] = variants and rng.random() < 0.5
    return c


def lengths(case):
    """New tokens and cached tokens (with the new ones) of each sequence; for
    ``branch`` none and the cached tokens of each prompt."""
    r = random.Random(case["lens"])
    if case["op"] == "branch":
        return None, [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["parents"])]
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    q[0] = max(1, q[0])
    kv = [max(n, r.randint(case["kv_lo"], case["kv_hi"])) for n in q]
    return q, kv


def _page_bytes(case):
    """A page's K and V codes and scales."""
    return case["hkv"] * 2 * (PAGE * DIM * (2 if case["cache"] == "bf16" else 1) + (4 if case["cache"] == "scaled" else 0))


def work(case):
    if case["op"] == "copy":
        n = case["count"] - case["count"] // 8
        return {"bytes": 2 * n * _page_bytes(case) + 8 * case["count"], "flops": 0}
    if case["op"] == "branch":
        _, kv = lengths(case)
        k, add = case["children"], case["add"]
        shared = sum(-(-s // PAGE) for s in kv)
        copied = sum(s % PAGE > 0 for s in kv) * k
        grown = sum(-(-(s + add) // PAGE) - s // PAGE for s in kv) * k
        # the rows that are freed and the rows that are read and written, their counts, every page's, and the copied pages
        return {"bytes": 4 * (k * shared + 2 * grown) + 4 * (1 + k) * shared + 16 * case["pool"] + 2 * copied * _page_bytes(case), "flops": 0}
    q, kv = lengths(case)
    hq, hkv, T = case["hq"], case["hkv"], sum(q)
    es = 2 if case["cache"] == "bf16" else 1
    if case["op"] == "norm_append":
        pages = sum(-(-s // PAGE) - (s - n) // PAGE for n, s in zip(q, kv) if n)
        b = T * hq * DIM * 4 + T * hkv * DIM * (4 + 2 * es) + T * case["rot"] * 4
        if case["cache"] == "scaled":
            b += pages * hkv * 2 * 8
        return {"bytes": b, "flops": T * (hq + hkv) * (4 * DIM + 3 * case["rot"])}
    read, pairs = 0, 0
    for n, s in zip(q, kv):
        w, f = case["window"], case["first"]
        if w < 0:
            read += s
            pairs += n * s - n * (n - 1) // 2
            continue
        lo = max(0, s - n - w)
        read += s - lo + min(f, lo)
        for p in range(s - n, s):
            lo = max(0, p - w)
            pairs += p + 1 - lo + min(f, lo)
    pg = -(-read // PAGE)
    return {"bytes": read * hkv * DIM * 2 * es + (pg * hkv * 8 if case["cache"] == "scaled" else 0) + T * hq * DIM * 4, "flops": 4 * pairs * hq * DIM}


# ---- inputs -------------------------------------------------------------------


def _cache(g, case, pages):
    """(codes, scales or None, descale or None) of a cache whose pages differ in size."""
    heads = case["hkv"]
    x = torch.randn(pages, PAGE, heads, DIM, device="cuda", generator=g)
    if case["cache"] == "bf16":
        return x.to(torch.bfloat16), None, None
    if case["cache"] == "e4m3":
        d = torch.empty(1, device="cuda").uniform_(0.02, 0.06, generator=g)
        return (x / d).clamp(-448, 448).to(FP8), None, d
    x *= torch.exp2(0.75 * torch.randn(pages, 1, heads, 1, device="cuda", generator=g))
    m, e = torch.frexp(x.abs().amax(dim=(1, 3)))
    s = torch.ldexp(torch.ones_like(m), e - 8 - (m <= 0.875).int())
    return (x / s[:, None, :, None]).clamp(-448, 448).to(FP8), s, None


def _caches(g, case, pages, st):
    for i in "01":
        st["cache" + i], st["scales" + i], st["descale" + i] = _cache(g, case, pages)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 1)
    st = dict(case=case)
    if case["op"] == "copy":
        _caches(g, case, case["pool"], st)
        n = case["count"]
        perm = torch.randperm(case["pool"], device="cuda", generator=g).to(torch.int32)
        st["src"], st["dst"] = perm[:n].contiguous(), perm[n:2 * n].contiguous()
        st["src"][7::8] = -1  # nothing to copy in these places
        st["dst"][7::8] = -1
        return st
    if case["op"] == "branch":
        return _prepare_branch(case, g, st)
    q, kv = lengths(case)
    T, B = sum(q), case["seqs"]
    npg = [-(-s // PAGE) for s in kv]
    pages = sum(npg) + 3
    perm = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    first = torch.tensor([sum(npg[:i]) for i in range(B)], dtype=torch.int64, device="cuda")
    count = torch.tensor(npg, dtype=torch.int64, device="cuda")
    col = torch.arange(max(npg), device="cuda")[None]
    st["table"] = perm[torch.where(col < count[:, None], first[:, None] + col, pages - 1)].contiguous()
    st["cu"] = torch.tensor([sum(q[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    st["used"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    st["max_q"] = max(max(q), 1)
    _caches(g, case, pages, st)
    hq, hkv = case["hq"], case["hkv"]

    def rnd(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if case["op"] == "chunk":
        st["q"] = rnd(T, hq, DIM).to(torch.bfloat16)
        st["out"] = torch.zeros(T, hq, DIM, dtype=torch.bfloat16, device="cuda")
        st["scale"] = DIM ** -0.5
        st["sinks"] = 2 * rnd(hq) if case["sinks"] else None
        return st
    half = case["rot"] // 2
    ang = torch.arange(max(kv), dtype=torch.float64, device="cuda")[:, None] * \
        10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
    dt = torch.bfloat16 if case["weights"] == "bf16" else torch.float32
    st["q_norm"], st["k_norm"] = ((1 - case["offset"] + 0.1 * rnd(DIM)).to(dt) for _ in range(2))
    # the projections' one output [T, (hq + 2 hkv) * 256], tokens of different sizes: q, k and v are views of it
    qkv = (torch.exp2(0.75 * rnd(T, 1, 1)) * rnd(T, hq + 2 * hkv, DIM)).to(torch.bfloat16)
    st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    st["q_out"] = torch.zeros(T, hq, DIM, dtype=torch.bfloat16, device="cuda")
    return st


def _prepare_branch(case, g, st):
    """Prompts in the first rows, their candidates behind them, as a round of
    sampling left them: each candidate shares its prompt's full pages and has
    pages of its own behind them."""
    _, kv = lengths(case)
    P, k, add, pool = case["parents"], case["children"], case["add"], case["pool"]
    r = random.Random(case["lens"] + 1)
    ids = list(range(pool))
    r.shuffle(ids)
    width = max(-(-(s + add) // PAGE) for s in kv) + 1
    table = torch.zeros(P * (1 + k), width, dtype=torch.int32)
    used, count, refs = [0] * (P * (1 + k)), [0] * (P * (1 + k)), torch.zeros(pool, dtype=torch.int32)
    at = 0
    for p, s in enumerate(kv):
        n = -(-s // PAGE)
        table[p, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        used[p], count[p] = s, n
        refs[table[p, :n].long()] += 1
        at += n
    for p, s in enumerate(kv):
        for c in range(P + p * k, P + (p + 1) * k):
            full, n = s // PAGE, -(-(s + add) // PAGE)
            table[c, :full] = table[p, :full]
            table[c, full:n] = torch.tensor(ids[at:at + n - full], dtype=torch.int32)
            used[c], count[c] = s + add // 2, n
            refs[table[c, :n].long()] += 1
            at += n - full
    st.update(table=table.cuda(), used=torch.tensor(used, dtype=torch.int32, device="cuda"),
              count=torch.tensor(count, dtype=torch.int32, device="cuda"), refs=refs.cuda())
    st["children"] = torch.arange(P, P * (1 + k), dtype=torch.int32, device="cuda")
    st["parents"] = torch.arange(P, device="cuda").repeat_interleave(k).to(torch.int32)
    st["add"] = torch.where(torch.arange(P * (1 + k), device="cuda") < P, 0, add).to(torch.int32)
    _caches(g, case, pool, st)
    return st


# ---- one pass -----------------------------------------------------------------


def run(st):
    if own:
        return _own(st)
    return {"chunk": _chunk, "norm_append": _norm_append, "branch": _branch, "copy": _copy_pass}[st["case"]["op"]](st)


def _own(st):
    import speculative_decoding_verify_split_gb300 as va
    c = st["case"]
    if c["op"] == "chunk":
        return va.verify_attn_chunk(st["q"], st["cache0"], st["cache1"], st["table"], st["cu"], st["used"], st["scale"], k_descale=st["descale0"],
                                    v_descale=st["descale1"], k_scales=st["scales0"], v_scales=st["scales1"], out=st["out"],
                                    window_left=c["window"], first_tokens=c["first"], softcap=c["softcap"], sinks=st["sinks"])
    if c["op"] == "norm_append":
        va.append_kv(st["k"], st["v"], st["cache0"], st["cache1"], st["table"], st["cu"], st["used"], q=st["q"], q_out=st["q_out"],
                     cos_sin=st["cos_sin"], interleaved=c["interleaved"], k_descale=st["descale0"], v_descale=st["descale1"],
                     k_scales=st["scales0"], v_scales=st["scales1"], q_norm=st["q_norm"], k_norm=st["k_norm"], norm_eps=1e-6,
                     norm_offset=c["offset"])
        return _written(st)
    if c["op"] == "copy":
        va.copy_pages(st["cache0"], st["cache1"], st["src"], st["dst"], k_scales=st["scales0"], v_scales=st["scales1"])
        return _written(st)
    va.free_pages(st["table"], st["used"], st["count"], st["refs"], st["children"])
    va.fork_pages(st["table"], st["used"], st["count"], st["refs"], st["parents"], st["children"])
    src, dst, room = va.reserve_pages(st["table"], st["used"], st["count"], st["refs"], st["add"])
    va.copy_pages(st["cache0"], st["cache1"], src, dst, k_scales=st["scales0"], v_scales=st["scales1"])
    return dict(_written(st), src=src, dst=dst, room=room)


def _written(st):
    return {k: st[k] for k in ("q_out", "cache0", "cache1", "scales0", "scales1", "table", "used", "count", "refs")
            if st.get(k) is not None and (k not in ("table", "used") or "refs" in st)}


def _tokens(st, T):
    """For each new token: its sequence, its number there and its position."""
    n = st["cu"][1:] - st["cu"][:-1]
    i = torch.arange(T, device="cuda")
    b = torch.searchsorted(st["cu"][1:], i, right=True)
    t = i - st["cu"][b]
    return b, t, st["used"][b] - n[b] + t


def _values(st, i):
    """The cache's values of every sequence, zero past its last token: [B, keys, heads, dim]."""
    table = st["table"].long()
    x = st["cache" + i][table].float()
    if st["scales" + i] is not None:
        x = x * st["scales" + i][table][:, :, None, :, None]
    if st["descale" + i] is not None:
        x = x * st["descale" + i]
    x = x.reshape(table.shape[0], -1, *x.shape[3:])
    return torch.where((torch.arange(x.shape[1], device="cuda")[None] < st["used"][:, None])[:, :, None, None], x, 0.0)


def _chunk(st):
    c = st["case"]
    K, V = _values(st, "0"), _values(st, "1")
    B, keys, hkv = K.shape[:3]
    group, L = c["hq"] // hkv, st["max_q"]
    b, t, pos = _tokens(st, st["q"].shape[0])
    q = torch.zeros(B, L, c["hq"], DIM, device="cuda")
    q[b, t] = st["q"].float()
    q = q.view(B, L, hkv, group, DIM).permute(0, 2, 3, 1, 4).reshape(B, hkv, group * L, DIM)
    s = (q @ K.permute(0, 2, 3, 1)).mul_(st["scale"]).view(B, c["hq"], L, keys)
    if c["softcap"]:
        s.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    n = st["cu"][1:] - st["cu"][:-1]
    at = ((st["used"] - n)[:, None] + torch.arange(L, device="cuda"))[:, :, None]  # position of token t
    key = torch.arange(keys, device="cuda")
    vis = (key <= at) & (key < st["used"][:, None, None])
    if c["window"] >= 0:
        vis &= (key >= at - c["window"]) | (key < c["first"])
    s.masked_fill_(~vis[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(top).exp_()
    den = p.sum(-1, keepdim=True)
    if st["sinks"] is not None:
        den = den + torch.exp(st["sinks"][:, None, None] - top)
    o = p.view(B, hkv, group * L, keys) @ V.permute(0, 2, 1, 3)
    o = torch.where(vis.any(-1)[:, None, :, None], o.view(B, c["hq"], L, DIM) / den, 0.0)
    return o.permute(0, 2, 1, 3)[b, t].to(torch.bfloat16)


def _normed(x, w, offset):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (w.float() + offset)


def _rotate(x, cos_sin, pos, interleaved):
    rot = cos_sin.shape[1]
    cos, sin = cos_sin[pos][:, None].chunk(2, dim=-1)
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        x1, x2 = head[..., 0::2], head[..., 1::2]
        y = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1).flatten(-2)
    else:
        x1, x2 = head.chunk(2, dim=-1)
        y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1)
    return torch.cat([y, rest], dim=-1)


def _bytes(x):
    return x.view(torch.uint8) if x.dtype == FP8 else x


def _store(st, x, i, b, pos):
    """Stores rows x [T, heads, dim] (32 bits) at positions pos of their sequences in cache i."""
    cache, scales, descale = st["cache" + i], st["scales" + i], st["descale" + i]
    page = st["table"][b, pos // PAGE].long()
    if cache.dtype == torch.bfloat16:
        cache[page, pos % PAGE] = x.to(torch.bfloat16)
        return
    if scales is None:
        _bytes(cache)[page, pos % PAGE] = _bytes((x / descale).clamp(-448, 448).to(FP8))
        return
    n = st["cu"][1:] - st["cu"][:-1]
    start = st["used"] - n                                   # position of each sequence's first new token
    page0 = st["table"].gather(1, (start // PAGE).clamp(max=st["table"].shape[1] - 1).long()[:, None])[:, 0].long()
    kept = torch.where(n > 0, start % PAGE, 0)               # older tokens of that page
    amax = torch.zeros_like(scales).scatter_reduce(0, page[:, None].expand(-1, scales.shape[1]), x.abs().amax(-1), "amax")
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 8 - (m <= 0.875).int(), -64).clamp(-64, 64)
    need = torch.ldexp(torch.ones_like(amax), e)
    had = torch.zeros_like(scales)
    had[page0] = torch.where(kept[:, None] > 0, scales[page0].clamp(2.0 ** -64, 2.0 ** 64), 0.0)
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda")
    touched[page] = True
    new = torch.where(touched[:, None], torch.maximum(had, need), scales)
    old = cache[page0].float() * had[page0][:, None, :, None]
    old = _bytes((old / new[page0][:, None, :, None]).clamp(-448, 448).to(FP8))
    keep = (torch.arange(PAGE, device="cuda")[None] < kept[:, None])[:, :, None, None]
    _bytes(cache)[page0] = torch.where(keep, old, _bytes(cache)[page0])
    _bytes(cache)[page, pos % PAGE] = _bytes((x / new[page][:, :, None]).clamp(-448, 448).to(FP8))
    scales.copy_(new)


def _norm_append(st):
    c = st["case"]
    b, t, pos = _tokens(st, st["k"].shape[0])
    st["q_out"].copy_(_rotate(_normed(st["q"], st["q_norm"], c["offset"]), st["cos_sin"], pos, c["interleaved"]))
    _store(st, _rotate(_normed(st["k"], st["k_norm"], c["offset"]), st["cos_sin"], pos, c["interleaved"]), "0", b, pos)
    _store(st, st["v"].float(), "1", b, pos)
    return _written(st)


def _copy(st, src, dst):
    m = (src >= 0) & (dst >= 0)
    a, z = src[m].long(), dst[m].long()
    _bytes(st["cache0"])[z] = _bytes(st["cache0"])[a]
    _bytes(st["cache1"])[z] = _bytes(st["cache1"])[a]
    if st["scales0"] is not None:
        st["scales0"][z] = st["scales0"][a]
        st["scales1"][z] = st["scales1"][a]


def _copy_pass(st):
    _copy(st, st["src"], st["dst"])
    return _written(st)


def _branch(st):
    table, used, count, refs = st["table"], st["used"], st["count"], st["refs"]
    width = table.shape[1]
    place = torch.arange(width, device="cuda")[None]
    par, chi = st["parents"].long(), st["children"].long()
    # free the last candidates
    refs.index_add_(0, table[chi].flatten().long(), -(place < count[chi][:, None]).flatten().int())
    used[chi] = 0
    count[chi] = 0
    # fork: the prompt's pages are the new candidate's too
    n = (used[par] + PAGE - 1) // PAGE
    mine = place < n[:, None]
    table[chi] = torch.where(mine, table[par], table[chi])
    refs.index_add_(0, table[par].flatten().long(), mine.flatten().int())
    used[chi] = used[par]
    count[chi] = n
    # room for the next tokens, in pages of the sequence's own
    want = (used + st["add"] + PAGE - 1) // PAGE
    write = (place >= (used // PAGE)[:, None]) & (place < want[:, None]) & (st["add"] > 0)[:, None] & (want <= width)[:, None]
    shared = write & (place < count[:, None]) & (refs[table.long()] > 1)
    need = shared | (write & (place >= count[:, None]))
    each = need.sum(1)
    free = (refs == 0).nonzero()[:, 0]
    ok = (want <= width) & (st["add"] > 0) & ((each == 0) | (each.cumsum(0) <= free.shape[0]))
    need, shared = need & ok[:, None], shared & ok[:, None]
    last = (used // PAGE).clamp(max=width - 1).long()[:, None]
    moved = shared.gather(1, last)[:, 0] & (used % PAGE > 0)
    src = torch.where(moved, table.gather(1, last)[:, 0], -1)
    refs.index_add_(0, table.flatten().long(), -shared.flatten().int())
    fresh = free[(need.flatten().cumsum(0) - 1).clamp(0, max(0, free.shape[0] - 1))].view_as(table).int()
    table.copy_(torch.where(need, fresh, table))
    refs[fresh[need].long()] = 1
    dst = torch.where(moved, table.gather(1, last)[:, 0], -1)
    count.copy_(torch.where(ok, torch.maximum(count, want), count))
    _copy(st, src, dst)
    return dict(_written(st), src=src, dst=dst, room=count * PAGE)


# ---- the definitions in 64 bits, sequence by sequence --------------------------


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "chunk":
        return _exact_chunk(st, *lengths(case))
    if case["op"] == "norm_append":
        return _exact_append(st, *lengths(case))
    return _exact_pool(st)


def _exact_chunk(st, q, kv):
    c = st["case"]
    group = c["hq"] // c["hkv"]
    out = torch.zeros(sum(q), c["hq"], DIM, dtype=torch.float64, device="cuda")

    def head(i, pages, h, s):
        x = st["cache" + i][pages, :, h].double()
        if st["scales" + i] is not None:
            x = x * st["scales" + i][pages, h].double()[:, None, None]
        if st["descale" + i] is not None:
            x = x * st["descale" + i].double()
        return x.flatten(0, 1)[:s]

    a = 0
    for i, (n, s) in enumerate(zip(q, kv)):
        pages = st["table"][i, :-(-s // PAGE)].long()
        row = torch.arange(s - n, s, device="cuda")[:, None]
        col = torch.arange(s, device="cuda")[None]
        hidden = col > row
        if c["window"] >= 0:
            hidden |= (row - col > c["window"]) & (col >= c["first"])
        for h in range(c["hkv"]):
            K, V = head("0", pages, h, s), head("1", pages, h, s)
            for j in range(h * group, (h + 1) * group):
                x = st["scale"] * (st["q"][a:a + n, j].double() @ K.T)
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                x.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(x, dim=1, keepdim=True)
                if st["sinks"] is not None:
                    z = torch.logaddexp(z, st["sinks"][j].double())
                out[a:a + n, j] = x.sub_(z).exp_() @ V
        a += n
    return out


def _turned(x, table, p0, interleaved):
    """Rows x [n, heads, dim] at positions p0, p0 + 1, ...: complex products."""
    rot = table.shape[1]
    ang = table[p0:p0 + x.shape[0]].double()
    w = torch.complex(ang[:, :rot // 2], ang[:, rot // 2:])[:, None]
    y = x.clone()
    if interleaved:
        z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous()) * w
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_append(st, q, kv):
    c = st["case"]
    table = st["table"].cpu()
    res = {k: st[k].double() for k in ("q_out", "cache0", "cache1", "scales0", "scales1") if st.get(k) is not None}
    a = 0
    for i, (n, s) in enumerate(zip(q, kv)):
        if not n:
            continue
        z = a + n

        def turned(x, w):
            x = x[a:z].double()
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / DIM + 1e-6) * (w.double() + c["offset"])
            return _turned(x, st["cos_sin"], s - n, c["interleaved"])

        res["q_out"][a:z] = turned(st["q"], st["q_norm"])
        for which, x in (("0", turned(st["k"], st["k_norm"])), ("1", st["v"][a:z].double())):
            cache, scales, de = res["cache" + which], res.get("scales" + which), st["descale" + which]
            p = s - n
            while p < s:
                page, lo = int(table[i, p // PAGE]), p % PAGE
                hi = min(PAGE, lo + s - p)
                new = x[p - (s - n):p - (s - n) + hi - lo]
                if scales is not None:
                    m, e = torch.frexp(new.abs().amax(dim=(0, 2)))
                    need = torch.exp2(torch.where(m > 0, e - torch.where(m <= 0.875, 9, 8), -64).clamp(-64, 64).double())
                    if lo:
                        had = scales[page].clone()
                        scales[page] = torch.maximum(had, need)
                        cache[page, :lo] *= (had / scales[page])[None, :, None]
                    else:
                        scales[page] = need
                    new = new / scales[page][None, :, None]
                elif de is not None:
                    new = (new / de.double()).clamp(-448, 448)
                cache[page, lo:hi] = new
                p += hi - lo
        a = z
    return res


def _exact_pool(st):
    """Page by page, as a program on the host would keep such a pool; what is copied has its own value."""
    c = st["case"]
    res = {k: st[k].double() for k in ("cache0", "cache1", "scales0", "scales1") if st.get(k) is not None}
    if c["op"] == "copy":
        moves = list(zip(st["src"].tolist(), st["dst"].tolist()))
        whole = {}
    else:
        table, used, count, refs = (st[k].tolist() for k in ("table", "used", "count", "refs"))
        for s in st["children"].tolist():
            for page in table[s][:count[s]]:
                refs[page] -= 1
            used[s] = count[s] = 0
        for p, s in zip(st["parents"].tolist(), st["children"].tolist()):
            n = -(-used[p] // PAGE)
            table[s][:n] = table[p][:n]
            for page in table[p][:n]:
                refs[page] += 1
            used[s], count[s] = used[p], n
        free = [i for i, r in enumerate(refs) if r == 0]
        before = list(refs)
        src, dst = [-1] * len(used), [-1] * len(used)
        wanted = 0
        for s, add in enumerate(st["add"].tolist()):
            want = -(-(used[s] + add) // PAGE)
            if add <= 0 or want > len(table[s]):
                continue
            places = [j for j in range(used[s] // PAGE, want) if j >= count[s] or before[table[s][j]] > 1]
            wanted += len(places)
            if places and wanted > len(free):
                continue
            for k, j in enumerate(places):
                page = free[wanted - len(places) + k]
                if j < count[s]:
                    refs[table[s][j]] -= 1
                    if j == used[s] // PAGE and used[s] % PAGE:
                        src[s], dst[s] = table[s][j], page
                refs[page] = 1
                table[s][j] = page
            count[s] = max(count[s], want)
        moves = list(zip(src, dst))
        whole = dict(table=table, used=used, count=count, refs=refs, src=src, dst=dst, room=[n * PAGE for n in count])
    for a, z in moves:
        if a >= 0:
            for x in res.values():
                x[z] = x[a]
    return dict(res, **{k: torch.tensor(v, dtype=torch.int32) for k, v in whole.items()})
