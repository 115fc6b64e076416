"""Refusals of verify_attn_chunk: status codes from the host checks, before any
launch (CPU tensors, C ABI called directly), and the binding's own checks; the
oracle against closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import descriptors
from oracle.chunk_fp64 import chunk_oracle

NULL, SHAPE, DTYPE, UNSUPPORTED, LAYOUT = 1, 2, 3, 4, 7
BF, F8, I = torch.bfloat16, torch.float8_e4m3fn, torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verify_split_gb300.build import build_library
    build_library()


def args(**kw):
    a = dict(q=torch.zeros(5, 4, 256, dtype=BF), k=torch.zeros(8, 16, 2, 256, dtype=BF), v=torch.zeros(8, 16, 2, 256, dtype=BF), ks=None, vs=None,
             bt=torch.zeros(2, 3, dtype=I), cu=torch.tensor([0, 2, 5], dtype=I), su=torch.tensor([4, 9], dtype=I), kd=None, vd=None,
             out=torch.zeros(5, 4, 256, dtype=BF), window=-1, softcap=0.0, sinks=None, first=0, splits=0, opts=True)
    a.update(kw)
    return a


def call(**kw):
    a = args(**kw)
    r = descriptors(a["q"], a["k"], a["v"], a["ks"], a["vs"], a["bt"], a["cu"], a["su"], a["kd"], a["vd"], a["out"])
    o = va.VaOptions(a["window"], a["softcap"], descriptors(a["sinks"])[0])
    return va.library().verify_attn_chunk(*r[:8], 0.0625, *r[8:], ctypes.pointer(o) if a["opts"] else None, a["first"], None, 0, a["splits"], None)


E = dict(k=torch.zeros(8, 16, 2, 256, dtype=torch.uint8).view(F8), v=torch.zeros(8, 16, 2, 256, dtype=torch.uint8).view(F8))
S = torch.ones(8, 2)
BAD = [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(bt=None), NULL), (dict(cu=None), NULL), (dict(su=None), NULL),
    (dict(out=None), NULL), (dict(E, ks=S), NULL), (dict(E, vs=S), NULL),
    (dict(q=torch.zeros(5, 1024, dtype=BF)), SHAPE), (dict(v=torch.zeros(7, 16, 2, 256, dtype=BF)), SHAPE),
    (dict(out=torch.zeros(5, 2, 256, dtype=BF)), SHAPE), (dict(q=torch.zeros(5, 3, 256, dtype=BF), out=torch.zeros(5, 3, 256, dtype=BF)), SHAPE),
    (dict(cu=torch.zeros(2, dtype=I)), SHAPE), (dict(bt=torch.zeros(3, 3, dtype=I)), SHAPE), (dict(E, ks=torch.ones(7, 2), vs=S), SHAPE),
    (dict(kd=torch.ones(2)), SHAPE), (dict(sinks=torch.zeros(3)), SHAPE),
    (dict(q=torch.zeros(5, 4, 256)), DTYPE), (dict(out=torch.zeros(5, 4, 256)), DTYPE), (dict(k=E["k"]), DTYPE), (dict(ks=S, vs=S), DTYPE),
    (dict(su=torch.zeros(2)), DTYPE), (dict(sinks=torch.zeros(4, dtype=BF)), DTYPE), (dict(E, ks=S.to(BF), vs=S), DTYPE),
    (dict(q=torch.zeros(5, 4, 128, dtype=BF), out=torch.zeros(5, 4, 128, dtype=BF)), UNSUPPORTED),
    (dict(k=torch.zeros(8, 32, 2, 256, dtype=BF), v=torch.zeros(8, 32, 2, 256, dtype=BF)), UNSUPPORTED),
    (dict(E, ks=S, vs=S, kd=torch.ones(1)), UNSUPPORTED), (dict(window=-2), UNSUPPORTED), (dict(softcap=-1.0), UNSUPPORTED),
    (dict(softcap=float("nan")), UNSUPPORTED), (dict(first=-1), UNSUPPORTED), (dict(splits=-1), UNSUPPORTED),
    (dict(q=torch.zeros(1, 4, 256, dtype=BF).expand(1 << 30, 4, 256), out=torch.zeros(5, 4, 256, dtype=BF)), SHAPE),
    (dict(out=torch.zeros(1, 4, 256, dtype=BF).expand(5, 4, 256)), LAYOUT),             # written rows on top of each other
    (dict(out=torch.zeros(5, 1, 256, dtype=BF).expand(5, 4, 256)), LAYOUT),
    (dict(q=torch.zeros(5, 4, 260, dtype=BF)[..., 4:]), LAYOUT), (dict(k=torch.zeros(8, 16, 2, 260, dtype=BF)[..., 2:258]), LAYOUT),
    (dict(su=torch.zeros(4, dtype=I)[::2]), LAYOUT), (dict(sinks=torch.zeros(8)[::2]), LAYOUT),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refuses(i):
    kw, code = BAD[i]
    assert call(**kw) == code


def test_too_many_rows():
    """total_q * Hq / Hkv past 31 bits."""
    big = torch.zeros(8, 256, dtype=BF).as_strided((1 << 27, 64, 256), (0, 0, 1))
    q, out = va.desc(big), va.desc(big)
    for i, n in enumerate((64 * 256, 256, 1)):
        out.stride[i] = n                    # (described, not there: the check comes first)
    r = descriptors(torch.zeros(8, 16, 1, 256, dtype=BF), torch.ones(8, 16, 1, 256, dtype=BF), torch.zeros(1, 3, dtype=I),
                    torch.zeros(2, dtype=I), torch.zeros(1, dtype=I))
    s = va.library().verify_attn_chunk(ctypes.byref(q), r[0], r[1], None, None, *r[2:], 1.0, None, None, ctypes.byref(out), None, 0, None, 0, 0, None)
    assert s == UNSUPPORTED


def test_no_rows_are_fine_without_a_gpu():
    e = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    assert call(q=e(0, 4, 256), out=e(0, 4, 256), cu=torch.zeros(3, dtype=I)) == 0
    assert call(bt=torch.zeros(0, 3, dtype=I), cu=torch.zeros(1, dtype=I), su=torch.zeros(0, dtype=I)) == 0
    assert call(q=e(0, 4, 256), out=e(0, 4, 256), cu=torch.zeros(3, dtype=I), opts=False) == 0


def test_binding_checks():
    a = args()
    base = (a["q"], a["k"], a["v"], a["bt"], a["cu"], a["su"], 0.0625)
    with pytest.raises(ValueError, match="CUDA"):
        va.verify_attn_chunk(*base, out=a["out"])
    with pytest.raises(TypeError):
        va.verify_attn_chunk(a["q"].half(), *base[1:], out=a["out"])
    with pytest.raises(ValueError, match="different devices"):
        va.verify_attn_chunk(*base, out=a["out"].to("meta"))
    with pytest.raises(OverflowError):
        va.verify_attn_chunk(*base, out=a["out"], first_tokens=1 << 40)


# ---- the oracle ---------------------------------------------------------------------------


def one(S, L, **kw):
    rng = np.random.default_rng(S + L)
    q, k, v = rng.standard_normal((L, 2, 8)), rng.standard_normal((4, 16, 1, 8)), rng.standard_normal((4, 16, 1, 8))
    table = np.array([[2, 0, 3]])
    out, _ = chunk_oracle(q, k, v, table, [0, L], [S], 0.4, **kw)
    return q, k[[2, 0, 3], :, 0].reshape(-1, 8), v[[2, 0, 3], :, 0].reshape(-1, 8), out


def test_oracle_is_attention():
    q, k, v, out = one(40, 6)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.tensor(q).permute(1, 0, 2), torch.tensor(k[:40]).expand(2, 40, 8), torch.tensor(v[:40]).expand(2, 40, 8), scale=0.4,
        attn_mask=torch.arange(40)[None] <= torch.arange(34, 40)[:, None])
    assert np.allclose(out, want.permute(1, 0, 2).numpy(), atol=1e-12)


def test_oracle_variants():
    q, k, v, out = one(40, 3, window_left=0)
    assert np.allclose(out, v[37:40, None].repeat(2, 1))                       # a window of the token itself
    *_, out = one(40, 3, window_left=0, first_tokens=40)
    assert np.allclose(out, one(40, 3)[3])                                     # every token is a first one
    q, k, v, out = one(40, 1, window_left=5, first_tokens=2)
    j = [0, 1] + list(range(34, 40))
    p = np.exp(0.4 * (k[j] @ q[0, 0]))
    assert np.allclose(out[0, 0], p @ v[j] / p.sum())
    *_, out = one(2, 4)
    assert (out[:2] == 0).all() and np.isfinite(out).all()                     # tokens before position 0
    assert np.allclose(one(30, 2, softcap=1e6)[3], one(30, 2)[3], atol=1e-9)
    assert (np.abs(one(30, 2, sinks=np.array([50.0, 50.0]))[3]) < 1e-6).all()  # a sink that takes all
