"""The paged-cache operators: what each computes, in plain torch, and the cases
they are measured on.

Four operators around the paged KV cache of target-verify attention (16-token
pages, head_dim 256, or latent rows of 512 + 64):

* ``append``: the new tokens' keys are rotated by their positions and stored,
  with the values, in the pages that hold those positions; the queries are
  rotated beside them. Caches: bf16, e4m3 with one descale a tensor, e4m3 with
  a power-of-two scale for each page and KV head.
* ``latent_append``: the same for rows [latent | rope key] of a latent cache.
* ``scaled``: verify attention over an e4m3 cache with a scale for each page
  and KV head.
* ``latent_scaled``: verify attention over a latent e4m3 cache with a scale
  for each page.

Token t of sequence b (L new tokens, S cached tokens with them) is at position
S - L + t. Page scales: a page whose first new token is its first slot starts
afresh; else it holds older tokens under the scale it has. The scale becomes
the larger of that one and the smallest 2^e (-64 <= e <= 64) with
max|new| <= 448 * 2^e, and where it grows the older codes are rounded to it.
Stored e4m3 values saturate at +-448.
"""
import math
import random

import torch

own = False

PAGE = 16
DIM = 256
LATENT, ROPE = 512, 64
FP8 = torch.float8_e4m3fn


# ---- cases --------------------------------------------------------------------


def listed():
    return [
        # one verify step of two users: the latency of a call with almost no work
        dict(name="append_tiny_bf16", op="append", lens=1, seqs=2, q_lo=2, q_hi=4, kv_lo=769, kv_hi=1024, hq=16, hkv=1,
             cache="bf16", rot=256, interleaved=False),
        # a verify step of a mid-size batch over a cache with page scales, partial rotation
        dict(name="append_verify_scaled", op="append", lens=2, seqs=64, q_lo=3, q_hi=3, kv_lo=513, kv_hi=4096, hq=16, hkv=1,
             cache="scaled", rot=64, interleaved=True),
        # a high-concurrency verify step, ragged draft counts, per-tensor descales
        dict(name="append_many_fp8", op="append", lens=3, seqs=256, q_lo=1, q_hi=4, kv_lo=64, kv_hi=1024, hq=8, hkv=1,
             cache="e4m3", rot=128, interleaved=False),
        # the prompts of a batch behind cached prefixes of odd length
        dict(name="append_prompt_scaled", op="append", lens=4, seqs=8, q_lo=513, q_hi=4096, kv_lo=700, kv_hi=5000, hq=32, hkv=2,
             cache="scaled", rot=256, interleaved=False),
        # a latent model's verify step
        dict(name="latent_append_verify_bf16", op="latent_append", lens=5, seqs=64, q_lo=3, q_hi=3, kv_lo=513, kv_hi=4096, hq=16, hkv=1,
             cache="bf16", rot=64, interleaved=True),
        # a latent model's prompts into a cache with page scales
        dict(name="latent_append_prompt_scaled", op="latent_append", lens=6, seqs=16, q_lo=513, q_hi=4096, kv_lo=700, kv_hi=5000, hq=16, hkv=1,
             cache="scaled", rot=64, interleaved=False),
        # the smallest verify call
        dict(name="scaled_tiny_verify", op="scaled", lens=7, seqs=2, q_lo=2, q_hi=4, kv_lo=769, kv_hi=1024, hq=16, hkv=1,
             window=-1, softcap=0.0, sinks=False),
        # single-token decoding with every variant of the attention on
        dict(name="scaled_single_variants", op="scaled", lens=8, seqs=32, q_lo=1, q_hi=1, kv_lo=513, kv_hi=16384, hq=32, hkv=2,
             window=1023, softcap=30.0, sinks=True),
        # a verify step at middling context
        dict(name="scaled_mid_context", op="scaled", lens=9, seqs=64, q_lo=3, q_hi=3, kv_lo=8192, kv_hi=32768, hq=16, hkv=1,
             window=-1, softcap=0.0, sinks=False),
        # the headline verify step: long context
        dict(name="scaled_long_context", op="scaled", lens=10, seqs=16, q_lo=4, q_hi=4, kv_lo=65536, kv_hi=131072, hq=16, hkv=1,
             window=-1, softcap=0.0, sinks=False),
        # the latent forms of the smallest and of the middling verify call
        dict(name="latent_scaled_tiny", op="latent_scaled", lens=11, seqs=2, q_lo=2, q_hi=4, kv_lo=769, kv_hi=1024, hq=16, hkv=1),
        dict(name="latent_scaled_mid_context", op="latent_scaled", lens=12, seqs=64, q_lo=3, q_hi=3, kv_lo=8192, kv_hi=32768, hq=16, hkv=1),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "append", "scaled", "scaled", "latent_append", "latent_scaled"])
    c = dict(op=op, lens=rng.randrange(1 << 30), hkv=1)
    if op in ("append", "latent_append"):
        c["cache"] = rng.choice(["bf16", "e4m3", "scaled", "scaled"])
        c["interleaved"] = rng.random() < 0.5
        if op == "append":
            c["hkv"] = rng.choice([1, 2, 3, 4])
            c["hq"] = c["hkv"] * rng.choice([1, 2, 4, 5, 8])
            c["rot"] = rng.choice([32, 64, 128, 192, 256])
        else:
            c["hq"] = rng.choice([1, 3, 8, 16, 32])
            c["rot"] = ROPE
        if rng.random() < 0.5:  # verify steps
            c["seqs"] = logint(1, 256)
            c["q_lo"] = rng.choice([0, 1, 1, 2])
            c["q_hi"] = rng.choice([2, 3, 4])
            c["kv_lo"] = rng.choice([4, 17, 300])
            c["kv_hi"] = logint(301, 4096)
        else:  # prompts
            c["seqs"] = rng.choice([1, 2, 3, 5, 8])
            c["q_hi"] = logint(17, 2048)
            c["q_lo"] = max(1, c["q_hi"] // rng.choice([1, 2, 7]))
            c["kv_lo"] = c["q_hi"] + rng.choice([0, 1, 100])
            c["kv_hi"] = c["kv_lo"] + logint(1, 2048)
        return c
    if op == "scaled":
        c["hkv"] = rng.choice([1, 1, 2, 4])
        group = rng.choice([1, 4, 5, 8, 16])
    else:
        group = rng.choice([3, 8, 16])
    c["hq"] = c["hkv"] * group
    c["q_lo"] = 1
    c["q_hi"] = rng.choice([1, 2, 4])
    c["kv_hi"] = logint(40, 65536)
    c["kv_lo"] = max(1, c["kv_hi"] // rng.choice([1, 2, 30]))
    c["seqs"] = max(1, min(logint(1, 128), (1 << 20) // (c["kv_hi"] * c["hkv"])))
    if op == "scaled":
        variants = rng.random() < 0.4
        c["window"] = rng.choice([-1, 63, 500, 4000]) if variants else -1
        c["softcap"] = rng.choice([0.0, 15.0, 30.0]) if variants else 0.0
        c["sinks"] = variants and rng.random() < 0.5
    return c


def lengths(case):
    """New tokens and cached tokens (with the new ones) of each sequence."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["seqs"])]
    q[0] = max(1, q[0])
    kv = [max(n, r.randint(case["kv_lo"], case["kv_hi"])) for n in q]
    return q, kv


def work(case):
    q, kv = lengths(case)
    hq, hkv, T = case["hq"], case["hkv"], sum(q)
    es = 2 if case.get("cache") == "bf16" else 1
    pages = sum(-(-s // PAGE) - (s - n) // PAGE for n, s in zip(q, kv) if n)
    if case["op"] == "append":
        b = T * hq * DIM * 4 + T * hkv * DIM * (4 + 2 * es) + T * case["rot"] * 4
        if case["cache"] == "scaled":
            b += pages * hkv * 2 * 8
        return {"bytes": b, "flops": 3 * T * (hq + hkv) * case["rot"]}
    if case["op"] == "latent_append":
        b = T * hq * ROPE * 4 + T * (LATENT + ROPE) * (2 + es) + T * ROPE * 4
        if case["cache"] == "scaled":
            b += pages * 8
        return {"bytes": b, "flops": 3 * T * (hq + 1) * ROPE}
    win = case.get("window", -1)
    seen = [min(s, n + win) if win >= 0 else s for n, s in zip(q, kv)]
    pg = sum(-(-s // PAGE) for s in seen)
    if case["op"] == "scaled":
        rows = sum(n * s for n, s in zip(q, seen)) * hq
        return {"bytes": sum(seen) * hkv * DIM * 2 + pg * hkv * 8 + T * hq * DIM * 4, "flops": 4 * rows * DIM}
    rows = sum(n * s for n, s in zip(q, seen)) * hq
    return {"bytes": sum(seen) * (LATENT + ROPE) + pg * 4 + T * hq * (2 * LATENT + ROPE) * 2,
            "flops": 2 * rows * (2 * LATENT + ROPE)}


# ---- inputs -------------------------------------------------------------------


def _paged(g, pages, heads, dim):
    """Codes and power-of-two page scales of a cache whose pages differ in size."""
    codes = torch.empty(pages, PAGE, heads, dim, dtype=FP8, device="cuda")
    scales = torch.empty(pages, heads, dtype=torch.float32, device="cuda")
    for a in range(0, pages, 1 << 14):
        n = min(1 << 14, pages - a)
        x = torch.randn(n, PAGE, heads, dim, device="cuda", generator=g)
        x *= torch.exp2(0.75 * torch.randn(n, 1, heads, 1, device="cuda", generator=g))
        m, e = torch.frexp(x.abs().amax(dim=(1, 3)))
        s = torch.ldexp(torch.ones_like(m), e - 8 - (m <= 0.875).int())
        codes[a:a + n] = (x / s[:, None, :, None]).clamp(-448, 448).to(FP8)
        scales[a:a + n] = s
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 1)
    q, kv = lengths(case)
    T, B = sum(q), case["seqs"]
    npg = [-(-s // PAGE) for s in kv]
    width = max(npg)
    pages = sum(npg) + 3
    perm = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    first = torch.tensor([sum(npg[:i]) for i in range(B)], dtype=torch.int64, device="cuda")
    count = torch.tensor(npg, dtype=torch.int64, device="cuda")
    col = torch.arange(width, device="cuda")[None]
    table = perm[torch.where(col < count[:, None], first[:, None] + col, pages - 1)].contiguous()
    cu = torch.tensor([sum(q[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    used = torch.tensor(kv, dtype=torch.int32, device="cuda")
    st = dict(case=case, table=table, cu=cu, used=used, max_q=max(max(q), 1), max_k=width * PAGE)

    def rnd(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    latent = case["op"].startswith("latent")
    hkv, dim = (1, LATENT + ROPE) if latent else (case["hkv"], DIM)
    if case["op"].endswith("append"):
        half = case["rot"] // 2
        ang = torch.arange(max(kv), dtype=torch.float64, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        size = torch.exp2(0.75 * rnd(T, 1, 1))
        if case["cache"] == "scaled":
            st["cache0"], st["scales0"] = _paged(g, pages, hkv, dim)
        else:
            x = rnd(pages, PAGE, hkv, dim)
            st["cache0"] = x.to(torch.bfloat16) if case["cache"] == "bf16" else x.to(FP8)
            if case["cache"] == "e4m3":
                st["descale0"] = torch.full((1,), 0.037, device="cuda")
        if latent:
            rows = (size * rnd(T, 1, dim)).to(torch.bfloat16)
            st["latent"], st["k_pe"] = rows[:, 0, :LATENT], rows[:, 0, LATENT:]
            st["q_pe"] = rnd(T, case["hq"], ROPE).to(torch.bfloat16)
            st["q_out"] = torch.zeros(T, case["hq"], dim, dtype=torch.bfloat16, device="cuda")[:, :, LATENT:]
            return st
        if case["cache"] == "scaled":
            st["cache1"], st["scales1"] = _paged(g, pages, hkv, dim)
        else:
            x = rnd(pages, PAGE, hkv, dim)
            st["cache1"] = x.to(torch.bfloat16) if case["cache"] == "bf16" else x.to(FP8)
            if case["cache"] == "e4m3":
                st["descale1"] = torch.full((1,), 0.021, device="cuda")
        # the projections' one output [T, (hq + 2 hkv) * 256]: q, k and v are views of it
        qkv = (torch.cat([torch.ones(T, case["hq"], 1, device="cuda"), size.expand(T, 2 * hkv, 1)], dim=1) *
               rnd(T, case["hq"] + 2 * hkv, DIM)).to(torch.bfloat16)
        st["q"], st["k"], st["v"] = qkv[:, :case["hq"]], qkv[:, case["hq"]:case["hq"] + hkv], qkv[:, case["hq"] + hkv:]
        st["q_out"] = torch.zeros(T, case["hq"], DIM, dtype=torch.bfloat16, device="cuda")
        return st
    st["q"] = rnd(T, case["hq"], dim).to(torch.bfloat16)
    st["cache0"], st["scales0"] = _paged(g, pages, hkv, dim)
    if latent:
        st["scale"] = (128 + ROPE) ** -0.5
        st["out"] = torch.zeros(T, case["hq"], LATENT, dtype=torch.bfloat16, device="cuda")
        return st
    st["cache1"], st["scales1"] = _paged(g, pages, hkv, dim)
    st["scale"] = DIM ** -0.5
    st["out"] = torch.zeros(T, case["hq"], DIM, dtype=torch.bfloat16, device="cuda")
    st["sinks"] = 2 * rnd(case["hq"]) if case["sinks"] else None
    return st


# ---- one pass -----------------------------------------------------------------


def run(st):
    if own:
        return _own(st)
    return {"append": _append, "latent_append": _latent_append, "scaled": _scaled, "latent_scaled": _latent_scaled}[st["case"]["op"]](st)


def _own(st):
    import speculative_decoding_verify_split_gb300 as va
    c = st["case"]
    if c["op"] == "append":
        va.append_kv(st["k"], st["v"], st["cache0"], st["cache1"], st["table"], st["cu"], st["used"], q=st["q"], q_out=st["q_out"],
                     cos_sin=st["cos_sin"], interleaved=c["interleaved"], k_descale=st.get("descale0"), v_descale=st.get("descale1"),
                     k_scales=st.get("scales0"), v_scales=st.get("scales1"))
        return _written(st)
    if c["op"] == "latent_append":
        va.append_mla(st["latent"], st["k_pe"], st["cache0"], st["table"], st["cu"], st["used"], q_pe=st["q_pe"], q_pe_out=st["q_out"],
                      cos_sin=st["cos_sin"], interleaved=c["interleaved"], descale=st.get("descale0"), scales=st.get("scales0"))
        return _written(st)
    if c["op"] == "scaled":
        return va.verify_attn_scaled(st["q"], st["cache0"], st["cache1"], st["scales0"], st["scales1"], st["table"], st["cu"], st["used"],
                                     st["max_q"], st["max_k"], st["scale"], out=st["out"], window_left=c["window"], softcap=c["softcap"],
                                     sinks=st["sinks"])
    return va.verify_attn_mla_scaled(st["q"], st["cache0"], st["scales0"], st["table"], st["cu"], st["used"], st["max_q"], st["max_k"],
                                     st["scale"], out=st["out"])


def _written(st):
    return {k: st[k] for k in ("q_out", "cache0", "cache1", "scales0", "scales1") if k in st}


def _tokens(st):
    """For each new token: its sequence, its number there and its position."""
    n = st["cu"][1:] - st["cu"][:-1]
    i = torch.arange(st["q_out" if "q_out" in st else "q"].shape[0], device="cuda")
    b = torch.searchsorted(st["cu"][1:], i, right=True)
    t = i - st["cu"][b]
    return b, t, st["used"][b] - n[b] + t


def _rotate(x, cos_sin, pos, interleaved):
    x = x.float()
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


def _store(st, x, cache, scales, descale, b, pos):
    """Stores rows x [T, heads, dim] (32 bits) at positions pos of their sequences."""
    page = st["table"][b, pos // PAGE].long()
    if cache.dtype == torch.bfloat16:
        cache[page, pos % PAGE] = x.to(torch.bfloat16)
        return
    if scales is None:
        cache.view(torch.uint8)[page, pos % PAGE] = (x / descale).clamp(-448, 448).to(FP8).view(torch.uint8)
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
    old = (old / new[page0][:, None, :, None]).clamp(-448, 448).to(FP8)
    slot = torch.arange(PAGE, device="cuda")
    keep = (slot[None] < kept[:, None])[:, :, None, None]
    cache.view(torch.uint8)[page0] = torch.where(keep, old.view(torch.uint8), cache.view(torch.uint8)[page0])
    cache.view(torch.uint8)[page, pos % PAGE] = (x / new[page][:, :, None]).clamp(-448, 448).to(FP8).view(torch.uint8)
    scales.copy_(new)


def _append(st):
    b, t, pos = _tokens(st)
    inter = st["case"]["interleaved"]
    st["q_out"].copy_(_rotate(st["q"], st["cos_sin"], pos, inter))
    _store(st, _rotate(st["k"], st["cos_sin"], pos, inter), st["cache0"], st.get("scales0"), st.get("descale0"), b, pos)
    _store(st, st["v"].float(), st["cache1"], st.get("scales1"), st.get("descale1"), b, pos)
    return _written(st)


def _latent_append(st):
    b, t, pos = _tokens(st)
    inter = st["case"]["interleaved"]
    st["q_out"].copy_(_rotate(st["q_pe"], st["cos_sin"], pos, inter))
    row = torch.cat([st["latent"].float()[:, None], _rotate(st["k_pe"][:, None], st["cos_sin"], pos, inter)], dim=-1)
    _store(st, row, st["cache0"], st.get("scales0"), st.get("descale0"), b, pos)
    return _written(st)


def _attend(st, K, V, window, softcap, sinks):
    """K [B, keys, hkv, dim], V [B, keys, hkv, width] in 32 bits; q as given."""
    c = st["case"]
    B, keys, hkv = K.shape[:3]
    group, L = c["hq"] // hkv, st["max_q"]
    b, t, pos = _tokens(st)
    q = torch.zeros(B, L, c["hq"], st["q"].shape[2], device="cuda")
    q[b, t] = st["q"].float()
    q = q.view(B, L, hkv, group, -1).permute(0, 2, 1, 3, 4).reshape(B, hkv, L * group, -1)
    s = st["scale"] * (q @ K.permute(0, 2, 3, 1))                        # [B, hkv, L * group, keys]
    if softcap:
        s = softcap * torch.tanh(s / softcap)
    n = st["cu"][1:] - st["cu"][:-1]
    at = (st["used"] - n)[:, None] + torch.arange(L, device="cuda")       # position of draft token t
    key = torch.arange(keys, device="cuda")
    vis = (key <= at[:, :, None]) & (key < st["used"][:, None, None])
    if window >= 0:
        vis &= key >= at[:, :, None] - window
    vis = vis[:, None, :, None].expand(B, 1, L, group, keys).reshape(B, 1, L * group, keys)
    s = torch.where(vis, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(s - top)
    den = p.sum(-1, keepdim=True)
    if sinks is not None:
        z = sinks.view(hkv, 1, group).expand(hkv, L, group).reshape(1, hkv, L * group, 1)
        den = den + torch.exp(z - top)
    o = torch.where(vis.any(-1, keepdim=True), (p @ V.permute(0, 2, 1, 3)) / den, 0.0)
    o = o.view(B, hkv, L, group, -1).permute(0, 2, 1, 3, 4).reshape(B, L, c["hq"], -1)
    return o[b, t].to(torch.bfloat16)


def _values(cache, scales, table, used):
    """The cache's values of every sequence, zero past its last token: [B, keys, heads, dim]."""
    x = cache[table.long()].float() * scales[table.long()][:, :, None, :, None]
    x = x.reshape(table.shape[0], -1, *cache.shape[2:])
    return torch.where((torch.arange(x.shape[1], device="cuda")[None] < used[:, None])[:, :, None, None], x, 0.0)


def _scaled(st):
    c = st["case"]
    K = _values(st["cache0"], st["scales0"], st["table"], st["used"])
    V = _values(st["cache1"], st["scales1"], st["table"], st["used"])
    return _attend(st, K, V, c["window"], c["softcap"], st["sinks"])


def _latent_scaled(st):
    K = _values(st["cache0"], st["scales0"], st["table"], st["used"])
    return _attend(st, K, K[..., :LATENT], -1, 0.0, None)


# ---- the definitions in 64 bits, sequence by sequence --------------------------


def exact(case, seed):
    st = prepare(case, seed)
    q, kv = lengths(case)
    if case["op"].endswith("append"):
        return _exact_append(st, q, kv)
    return _exact_attention(st, q, kv)


def _turned(x, table, p0, interleaved):
    """Rows x [n, heads, dim] at positions p0, p0 + 1, ...: complex products."""
    rot = table.shape[1]
    ang = table[p0:p0 + x.shape[0]].double()
    w = torch.complex(ang[:, :rot // 2], ang[:, rot // 2:])[:, None]
    y = x.double().clone()
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
    res = {k: st[k].double() for k in ("q_out", "cache0", "cache1", "scales0", "scales1") if k in st}
    a = 0
    for i, (n, s) in enumerate(zip(q, kv)):
        if not n:
            continue
        z = a + n
        if c["op"] == "append":
            res["q_out"][a:z] = _turned(st["q"][a:z], st["cos_sin"], s - n, c["interleaved"])
            rows = {"0": _turned(st["k"][a:z], st["cos_sin"], s - n, c["interleaved"]), "1": st["v"][a:z].double()}
        else:
            res["q_out"][a:z] = _turned(st["q_pe"][a:z], st["cos_sin"], s - n, c["interleaved"])
            rows = {"0": torch.cat([st["latent"][a:z, None].double(), _turned(st["k_pe"][a:z, None], st["cos_sin"], s - n, c["interleaved"])], -1)}
        for which, x in rows.items():
            cache, scales, de = res["cache" + which], res.get("scales" + which), st.get("descale" + which)
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


def _exact_attention(st, q, kv):
    c = st["case"]
    latent = c["op"] == "latent_scaled"
    hkv = c["hkv"]
    group = c["hq"] // hkv
    out = torch.zeros(sum(q), c["hq"], LATENT if latent else DIM, dtype=torch.float64, device="cuda")
    win, cap = c.get("window", -1), c.get("softcap", 0.0)
    a = 0
    for i, (n, s) in enumerate(zip(q, kv)):
        pages = st["table"][i, :-(-s // PAGE)].long()
        for h in range(hkv):
            K = (st["cache0"][pages, :, h].double() * st["scales0"][pages, h].double()[:, None, None]).flatten(0, 1)[:s]
            V = K[:, :LATENT] if latent else \
                (st["cache1"][pages, :, h].double() * st["scales1"][pages, h].double()[:, None, None]).flatten(0, 1)[:s]
            for t in range(n):
                hi = s - n + t + 1
                lo = max(0, hi - 1 - win) if win >= 0 else 0
                rows = st["q"][a + t, h * group:(h + 1) * group].double()
                x = st["scale"] * (rows @ K[lo:hi].T)
                if cap:
                    x = cap * torch.tanh(x / cap)
                z = torch.logsumexp(x, dim=1, keepdim=True)
                if st.get("sinks") is not None:
                    z = torch.logaddexp(z, st["sinks"][h * group:(h + 1) * group, None].double())
                out[a + t, h * group:(h + 1) * group] = torch.exp(x - z) @ V[lo:hi]
        a += n
    return out
