"""The calls as a decoder makes them: a prompt appended in chunks, then verify
steps that append drafts, attend, take back what was refused, and go on, over
every kind of cache."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import decode, table
from oracle.attention_fp64 import softmax_attend
from oracle.page_scaled_fp64 import page_scaled_oracle
from parity_gate import check_gates

pytestmark = pytest.mark.gpu


class Decoder:
    """Sequences in one cache, with what each has been fed (fp64) kept beside."""

    def __init__(self, kind, latent, hq, hkv, seed):
        self.kind, self.latent, self.hq, self.hkv = kind, latent, hq, hkv
        self.g = torch.Generator().manual_seed(seed)
        self.B, self.width, self.pages = 3, 24, 80
        self.dim = 576 if latent else 256
        dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
        shape = (self.pages, 16, 1 if latent else hkv, self.dim)
        nan = torch.full(shape, float("nan")).to(dt).cuda()
        self.cache = [nan, nan.clone()]
        self.scales = [torch.full(shape[::2][:2], float("nan"), device="cuda") for _ in range(2)] if kind == "scaled" else [None, None]
        self.descale = [torch.tensor([0.03], device="cuda"), torch.tensor([0.05], device="cuda")] if kind == "e4m3" else [None, None]
        self.bt = torch.randperm(self.pages, generator=self.g)[:self.B * self.width].reshape(self.B, self.width).int().cuda()
        self.len = [0] * self.B
        self.cos_sin = table(400, 64 if latent else 128).cuda()
        self.scale = self.dim ** -0.5
        self.fed = [[] for _ in range(self.B)]     # per sequence: rows of (k, v) in fp64, after the rotation

    def rnd(self, *s):
        return torch.randn(*s, generator=self.g).to(torch.bfloat16).cuda()

    def rot(self, x, pos):
        """fp64 rotation by halves of x [n, heads, dim] at positions pos."""
        n = self.cos_sin.shape[1] // 2
        c, s = self.cos_sin.cpu().double()[pos][:, None, :n], self.cos_sin.cpu().double()[pos][:, None, n:]
        y = x.cpu().double().clone()
        o = 512 if self.latent else 0
        a, b = y[..., o:o + n].clone(), y[..., o + n:o + 2 * n].clone()
        y[..., o:o + n], y[..., o + n:o + 2 * n] = a * c - b * s, b * c + a * s
        return y

    def step(self, news, attend):
        T = sum(news)
        pos = torch.cat([torch.arange(l, l + n) for l, n in zip(self.len, news)])
        cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32).cuda()
        self.len = [l + n for l, n in zip(self.len, news)]
        used = torch.tensor(self.len, dtype=torch.int32).cuda()
        q = self.rnd(T, self.hq, self.dim)
        if self.latent:
            row = self.rnd(T, 576)
            k = self.rot(row[:, None], pos)
            v = k[..., :512]
            qr = self.rot(q, pos)
            va.append_mla(row[:, :512], row[:, 512:], self.cache[0], self.bt, cu, used, q_pe=q[..., 512:], q_pe_out=q[..., 512:],
                          cos_sin=self.cos_sin, descale=self.descale[0], scales=self.scales[0])
        else:
            qkv = self.rnd(T, self.hq + 2 * self.hkv, 256)
            qkv[:, :self.hq] = q
            q = qkv[:, :self.hq]
            k, v = qkv[:, self.hq:self.hq + self.hkv], qkv[:, self.hq + self.hkv:]
            qr = self.rot(q, pos)
            va.append_kv(k, v, *self.cache, self.bt, cu, used, q=q, q_out=q, cos_sin=self.cos_sin, k_descale=self.descale[0],
                         v_descale=self.descale[1], k_scales=self.scales[0], v_scales=self.scales[1])
            k, v = self.rot(k, pos), v.cpu().double()
        for b in range(self.B):
            a, z = int(cu[b]), int(cu[b + 1])
            self.fed[b] += [(k[i].numpy(), v[i].numpy()) for i in range(a, z)]
        if not attend:
            return
        mk = self.width * 16
        if self.latent and self.kind == "scaled":
            out = va.verify_attn_mla_scaled(q, self.cache[0], self.scales[0], self.bt, cu, used, max(news), mk, self.scale)
        elif self.latent:
            out = va.verify_attn_mla(q, self.cache[0], self.bt, cu, used, max(news), mk, self.scale, self.descale[0], self.descale[0])
        elif self.kind == "scaled":
            out = va.verify_attn_scaled(q, *self.cache, *self.scales, self.bt, cu, used, max(news), mk, self.scale)
        else:
            out = va.verify_attn(q, *self.cache, self.bt, cu, used, max(news), mk, self.scale, *self.descale)
        self.check(out, q, qr, cu, used, news)

    def check(self, out, q, qr, cu, used, news):
        got = out.double().cpu().numpy()
        # on the bytes of the cache, exactly what the attention promises
        c = [np.nan_to_num(decode(x.cpu())) for x in self.cache]
        if self.latent:
            c[1] = c[0][..., :512]
        s = [x.cpu().numpy() if x is not None else np.full((self.pages, c[0].shape[2]), 1.0 if d is None else float(d))
             for x, d in zip(self.scales, self.descale)]
        if self.latent:
            s[1] = s[0]
        ref, tol = page_scaled_oracle(decode(q.cpu()), c[0], c[1], s[0], s[1], self.bt.cpu().numpy(), cu.cpu().numpy(), used.cpu().numpy(), self.scale)
        assert (np.abs(got - ref) <= tol).all()
        check_gates(got, ref)
        # and near the attention of what was fed: bf16 keys and values within
        # 2^-8, e4m3 ones within 2^-4 of each, so the weighted sums within a
        # few times that of the rows' own size
        G = self.hq // self.hkv
        num = den = 0.0
        for b in range(self.B):
            K = np.stack([x[0] for x in self.fed[b]])
            V = np.stack([x[1] for x in self.fed[b]])
            a, z = int(cu[b]), int(cu[b + 1])
            vis = np.arange(z - a) + self.len[b] - (z - a) + 1
            for h in range(self.hq):
                want = softmax_attend(qr[a:z, h].numpy(), K[:, h // G], V[:, h // G], vis, self.scale)
                num += ((got[a:z, h] - want) ** 2).sum()
                den += (want ** 2).sum()
        assert np.sqrt(num / den) <= (2.0 ** -6 if self.kind == "bf16" else 2.0 ** -2)

    def take_back(self, counts):
        for b, n in enumerate(counts):
            self.len[b] -= n
            del self.fed[b][len(self.fed[b]) - n:]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "scaled"])
@pytest.mark.parametrize("latent", [False, True])
def test_prompt_then_verify_steps(kind, latent):
    d = Decoder(kind, latent, 8, 1 if latent else 2, 600)
    d.step([37, 100, 5], False)                    # prompts in two chunks, the second mid-page
    d.step([20, 1, 60], False)
    for k in range(6):
        d.step([4, 2 + k % 3, 1 + k % 4], True)
        d.take_back([k % 4, (k + 1) % 2, 0])       # refused drafts


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("B", [1, 3, 40])
def test_decoding_without_a_pause(latent, B):
    """Steps of one token each, append and attention queued back to back with no
    synchronisation (each kernel may start while the one before it ends): the
    bits of the same steps with a pause after every call."""
    g = torch.Generator().manual_seed(7)
    steps, dim, width = 50, 576 if latent else 256, 8
    size = torch.exp2(4 * torch.rand(steps, 1, 1, 1, generator=g) - 2)       # so that page scales grow on the way
    kv = (size * torch.randn(steps, 2, B, dim, generator=g)).to(torch.bfloat16).cuda()
    q0 = torch.randn(steps, B, 16, dim, generator=g).to(torch.bfloat16).cuda()
    bt = torch.randperm(B * width, generator=g).int().reshape(B, width).cuda()
    cu = torch.arange(B + 1, dtype=torch.int32).cuda()
    used = [torch.full((B,), 30 + i, dtype=torch.int32).cuda() for i in range(steps)]
    cos_sin = table(128, 64 if latent else 256).cuda()
    big = torch.zeros(1 << 28, device="cuda")

    def run(pause):
        cache = [torch.zeros(B * width, 16, 1, dim, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.full((B * width, 1), 2.0 ** -12, device="cuda") for _ in range(2)]
        outs = [torch.zeros(B, 16, 512 if latent else 256, dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
        q = q0.clone()
        torch.cuda.synchronize()
        if not pause:
            for _ in range(8):
                big.add_(1)                       # the launches queue up behind it
        for i in range(steps):
            if latent:
                va.append_mla(kv[i, 0][:, :512], kv[i, 0][:, 512:], cache[0], bt, cu, used[i], q_pe=q[i][..., 512:],
                              q_pe_out=q[i][..., 512:], cos_sin=cos_sin, scales=scales[0])
            else:
                va.append_kv(kv[i, 0][:, None], kv[i, 1][:, None], *cache, bt, cu, used[i], q=q[i], q_out=q[i], cos_sin=cos_sin,
                             k_scales=scales[0], v_scales=scales[1])
            if pause:
                torch.cuda.synchronize()
            if latent:
                va.verify_attn_mla_scaled(q[i], cache[0], scales[0], bt, cu, used[i], 1, width * 16, dim ** -0.5, out=outs[i])
            else:
                va.verify_attn_scaled(q[i], *cache, *scales, bt, cu, used[i], 1, width * 16, dim ** -0.5, out=outs[i])
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs, cache, scales

    a, b = run(True), run(False)
    assert all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a[1], b[1]))
    assert all(torch.equal(x, y) for x, y in zip(a[2], b[2]))
    assert not torch.equal(a[0][0], a[0][-1]) and a[0][-1].any()


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("latent", [False, True])
def test_outputs_made_for_another_stream(latent, handle):
    """Outputs that the calls create on a given stream, dropped at once while the
    current stream allocates and fills memory of the same size: no result of a
    kept call changes."""
    d = Decoder("scaled", latent, 8, 1 if latent else 2, 700)
    d.step([37, 100, 5], False)
    used = torch.tensor(d.len, dtype=torch.int32).cuda()
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32).cuda()
    q = d.rnd(3, 8, d.dim)
    s = torch.cuda.Stream()
    arg = s.cuda_stream if handle else s
    torch.cuda.synchronize()

    def call(stream):
        if latent:
            return va.verify_attn_mla_scaled(q, d.cache[0], d.scales[0], d.bt, cu, used, 1, d.width * 16, d.scale, stream=stream)
        return va.verify_attn_scaled(q, *d.cache, *d.scales, d.bt, cu, used, 1, d.width * 16, d.scale, stream=stream)

    ref = call(None).clone()
    kept = []
    for i in range(40):
        out = call(arg)
        if i % 2:
            kept.append(out)
        del out
        torch.empty_like(ref).fill_(float("nan"))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in kept)
    row = d.rnd(3, 1, 576)
    kv = [d.rnd(3, 2, 256) for _ in range(2)]
    for st in (None, arg):
        cache, scales = [c.clone() for c in d.cache], [x.clone() for x in d.scales]
        torch.cuda.synchronize()
        if latent:
            r = va.append_mla(row[:, 0, :512], row[:, 0, 512:], cache[0], d.bt, cu, used, q_pe=q[..., 512:], cos_sin=d.cos_sin,
                              scales=scales[0], stream=st)
        else:
            r = va.append_kv(*kv, *cache, d.bt, cu, used, q=q, cos_sin=d.cos_sin, k_scales=scales[0], v_scales=scales[1], stream=st)
        torch.cuda.synchronize()
        first = r.clone() if st is None else first
        assert torch.equal(r, first)


@pytest.mark.parametrize("latent", [False, True])
def test_a_captured_decoding_step(latent):
    """Append and attention captured once, replayed token after token with the
    lengths advanced on the device: the eager steps' bits."""
    g = torch.Generator().manual_seed(8)
    B, steps, dim, width = 5, 40, 576 if latent else 256, 6
    kv = torch.randn(steps, 2, B, dim, generator=g).to(torch.bfloat16).cuda()
    q0 = torch.randn(steps, B, 16, dim, generator=g).to(torch.bfloat16).cuda()
    bt = torch.randperm(B * width, generator=g).int().reshape(B, width).cuda()
    cu = torch.arange(B + 1, dtype=torch.int32).cuda()
    start = torch.tensor([1, 15, 16, 17, 33], dtype=torch.int32).cuda()
    cos_sin = table(128, 64 if latent else 256).cuda()

    def state():
        return dict(cache=[torch.zeros(B * width, 16, 1, dim, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)],
                    scales=[torch.ones(B * width, 1, device="cuda") for _ in range(2)], used=start.clone(), q=q0[0].clone(),
                    kv=kv[0].clone(), out=torch.zeros(B, 16, 512 if latent else 256, dtype=torch.bfloat16, device="cuda"))

    def step(t):
        if latent:
            va.append_mla(t["kv"][0, :, :512], t["kv"][0, :, 512:], t["cache"][0], bt, cu, t["used"], q_pe=t["q"][..., 512:],
                          q_pe_out=t["q"][..., 512:], cos_sin=cos_sin, scales=t["scales"][0])
            va.verify_attn_mla_scaled(t["q"], t["cache"][0], t["scales"][0], bt, cu, t["used"], 1, width * 16, dim ** -0.5, out=t["out"])
        else:
            va.append_kv(t["kv"][0][:, None], t["kv"][1][:, None], *t["cache"], bt, cu, t["used"], q=t["q"], q_out=t["q"],
                         cos_sin=cos_sin, k_scales=t["scales"][0], v_scales=t["scales"][1])
            va.verify_attn_scaled(t["q"], *t["cache"], *t["scales"], bt, cu, t["used"], 1, width * 16, dim ** -0.5, out=t["out"])
        t["used"] += 1

    e, r = state(), state()
    want = []
    for i in range(steps):
        e["q"].copy_(q0[i])
        e["kv"].copy_(kv[i])
        step(e)
        want.append(e["out"].clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(r)
    r["used"].copy_(start)
    for i in range(steps):
        r["q"].copy_(q0[i])
        r["kv"].copy_(kv[i])
        graph.replay()
        assert torch.equal(r["out"], want[i]), i
    for x, y in zip(e["cache"] + e["scales"], r["cache"] + r["scales"]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_calls_from_several_threads():
    """Four threads with a stream each decode their own sequences at the same time."""
    from concurrent.futures import ThreadPoolExecutor
    base = Decoder("scaled", False, 8, 2, 710)
    base.step([37, 100, 5], False)
    torch.cuda.synchronize()
    cu = torch.tensor([0, 2, 4, 6], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(9)
    new = torch.randn(4, 20, 6, 12, 256, generator=g).to(torch.bfloat16).cuda()

    def decode(i):
        cache, scales = [c.clone() for c in base.cache], [x.clone() for x in base.scales]
        used = [torch.tensor([n + 2 * (k + 1) for n in base.len], dtype=torch.int32).cuda() for k in range(20)]
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        outs = []
        with torch.cuda.stream(s):
            for k in range(20):
                x = new[i, k]
                q = va.append_kv(x[:, 8:10], x[:, 10:], *cache, base.bt, cu, used[k], q=x[:, :8], cos_sin=base.cos_sin,
                                 k_scales=scales[0], v_scales=scales[1])
                outs.append(va.verify_attn_scaled(q, *cache, *scales, base.bt, cu, used[k], 2, base.width * 16, base.scale))
            s.synchronize()
        return torch.stack(outs)

    want = [decode(i) for i in range(4)]
    with ThreadPoolExecutor(4) as ex:
        for _ in range(3):
            got = list(ex.map(decode, range(4)))
            assert all(torch.equal(a, b) for a, b in zip(got, want))
