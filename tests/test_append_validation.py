"""Refusals of the append calls: status codes from the host checks, before any
launch (CPU tensors, C ABI called directly), and the binding's own checks. The
oracle's rotation and scale rule are pinned to facts outside it."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from oracle.append_fp64 import append_oracle, page_scale, rotated, usable
from append_util import descriptors, rope_of, table

NULL, SHAPE, DTYPE, UNSUPPORTED, LAYOUT = 1, 2, 3, 4, 7


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verify_split_gb300.build import build_library
    build_library()


def kv_args(**kw):
    a = dict(q=torch.zeros(5, 4, 256, dtype=torch.bfloat16), k=torch.zeros(5, 2, 256, dtype=torch.bfloat16),
             v=torch.zeros(5, 2, 256, dtype=torch.bfloat16), bt=torch.zeros(2, 3, dtype=torch.int32),
             cu=torch.tensor([0, 2, 5], dtype=torch.int32), su=torch.tensor([4, 9], dtype=torch.int32),
             cos_sin=torch.zeros(64, 128), positions=None, interleaved=0, kd=None, vd=None, ks=None, vs=None,
             q_out=torch.zeros(5, 4, 256, dtype=torch.bfloat16), kc=torch.zeros(8, 16, 2, 256, dtype=torch.bfloat16),
             vc=torch.zeros(8, 16, 2, 256, dtype=torch.bfloat16))
    a.update(kw)
    return a


def call_kv(**kw):
    a = kv_args(**kw)
    r = descriptors(a["q"], a["k"], a["v"], a["bt"], a["cu"], a["su"], a["kd"], a["vd"], a["ks"], a["vs"], a["q_out"], a["kc"], a["vc"])
    return va.library().verify_attn_append_kv(*r[:6], rope_of(a["cos_sin"], a["positions"], a["interleaved"]), *r[6:], None)


def call_mla(**kw):
    a = dict(q=torch.zeros(5, 4, 64, dtype=torch.bfloat16), latent=torch.zeros(5, 512, dtype=torch.bfloat16),
             k_pe=torch.zeros(5, 64, dtype=torch.bfloat16), bt=torch.zeros(2, 3, dtype=torch.int32),
             cu=torch.tensor([0, 2, 5], dtype=torch.int32), su=torch.tensor([4, 9], dtype=torch.int32),
             cos_sin=torch.zeros(64, 64), positions=None, interleaved=0, descale=None, scales=None,
             q_out=torch.zeros(5, 4, 64, dtype=torch.bfloat16), kc=torch.zeros(8, 16, 1, 576, dtype=torch.bfloat16))
    a.update(kw)
    r = descriptors(a["q"], a["latent"], a["k_pe"], a["bt"], a["cu"], a["su"], a["descale"], a["scales"], a["q_out"], a["kc"])
    return va.library().verify_attn_append_mla(*r[:6], rope_of(a["cos_sin"], a["positions"], a["interleaved"]), *r[6:], None)


BF, F8 = torch.bfloat16, torch.float8_e4m3fn
E4 = dict(kc=torch.zeros(8, 16, 2, 256, dtype=torch.uint8).view(F8), vc=torch.zeros(8, 16, 2, 256, dtype=torch.uint8).view(F8))
S82 = torch.ones(8, 2)
ONE = torch.zeros(8, 16, 2, 256, dtype=BF)

KV_BAD = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(bt=None), NULL), (dict(cu=None), NULL), (dict(su=None), NULL),
    (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(q=None), NULL), (dict(q_out=None), NULL),
    (dict(cos_sin=None), NULL),                                                         # q without a rotation
    (dict(E4, ks=S82), NULL), (dict(E4, vs=S82), NULL),                                 # one of the scales alone
    (dict(k=torch.zeros(5, 512, dtype=BF)), SHAPE), (dict(v=torch.zeros(4, 2, 256, dtype=BF)), SHAPE),
    (dict(k=torch.zeros(5, 3, 256, dtype=BF), v=torch.zeros(5, 3, 256, dtype=BF)), SHAPE),   # heads unlike the cache's
    (dict(vc=torch.zeros(7, 16, 2, 256, dtype=BF)), SHAPE), (dict(cu=torch.zeros(2, dtype=torch.int32)), SHAPE),
    (dict(bt=torch.zeros(3, 3, dtype=torch.int32)), SHAPE), (dict(q=torch.zeros(4, 4, 256, dtype=BF)), SHAPE),
    (dict(q_out=torch.zeros(5, 3, 256, dtype=BF)), SHAPE), (dict(cos_sin=torch.zeros(64)), SHAPE),
    (dict(cos_sin=torch.zeros(0, 64)), SHAPE), (dict(positions=torch.zeros(4, dtype=torch.int32)), SHAPE),
    (dict(E4, ks=torch.ones(7, 2), vs=S82), SHAPE), (dict(E4, ks=torch.ones(8), vs=S82), SHAPE),
    (dict(kd=torch.ones(2)), SHAPE),
    (dict(k=torch.zeros(5, 2, 256)), DTYPE), (dict(q=torch.zeros(5, 4, 256)), DTYPE), (dict(kc=torch.zeros(8, 16, 2, 256)), DTYPE),
    (dict(kc=E4["kc"]), DTYPE), (dict(ks=S82, vs=S82), DTYPE),                          # scales over a bf16 cache
    (dict(E4, ks=S82.to(BF), vs=S82), DTYPE), (dict(cos_sin=torch.zeros(64, 128, dtype=BF)), DTYPE),
    (dict(positions=torch.zeros(5)), DTYPE), (dict(su=torch.zeros(2)), DTYPE), (dict(kd=torch.ones(1, dtype=BF)), DTYPE),
    (dict(k=torch.zeros(5, 2, 128, dtype=BF), v=torch.zeros(5, 2, 128, dtype=BF)), UNSUPPORTED),
    (dict(q=torch.zeros(5, 4, 128, dtype=BF), q_out=torch.zeros(5, 4, 128, dtype=BF)), UNSUPPORTED),
    (dict(kc=torch.zeros(8, 32, 2, 256, dtype=BF), vc=torch.zeros(8, 32, 2, 256, dtype=BF)), UNSUPPORTED),
    (dict(cos_sin=torch.zeros(64, 4)), UNSUPPORTED), (dict(cos_sin=torch.zeros(64, 20)), UNSUPPORTED),
    (dict(cos_sin=torch.zeros(64, 264)), UNSUPPORTED), (dict(interleaved=2), UNSUPPORTED),
    (dict(E4, ks=S82, vs=S82, kd=torch.ones(1)), UNSUPPORTED),
    (dict(q=torch.zeros(5, 262200, 1, dtype=BF).expand(5, 262200, 256)), SHAPE),
    (dict(k=torch.zeros(5, 2, 260, dtype=BF)[:, :, 2:258]), LAYOUT), (dict(k=torch.zeros(256, 2, 5, dtype=BF).permute(2, 1, 0)), LAYOUT),
    (dict(q_out=torch.zeros(1, 4, 256, dtype=BF).expand(5, 4, 256)), LAYOUT),           # written rows on top of each other
    (dict(kc=torch.zeros(1, 16, 2, 256, dtype=BF).expand(8, 16, 2, 256)), LAYOUT),
    (dict(E4, ks=torch.ones(1, 2).expand(8, 2), vs=S82), LAYOUT), (dict(E4, ks=S82, vs=torch.ones(8, 1).expand(8, 2)), LAYOUT),
    (dict(cos_sin=torch.zeros(64, 130)[:, :128]), LAYOUT), (dict(positions=torch.zeros(10, dtype=torch.int32)[::2]), LAYOUT),
    (dict(su=torch.zeros(4, dtype=torch.int32)[::2]), LAYOUT),
    (dict(kc=ONE, vc=ONE), LAYOUT), (dict(E4, ks=S82, vs=S82), LAYOUT),                 # K and V in one place
]


@pytest.mark.parametrize("i", range(len(KV_BAD)))
def test_append_kv_refuses(i):
    kw, code = KV_BAD[i]
    assert call_kv(**kw) == code


MLA_BAD = [
    (dict(latent=None), NULL), (dict(k_pe=None), NULL), (dict(kc=None), NULL), (dict(q=None), NULL), (dict(q_out=None), NULL),
    (dict(cos_sin=None), NULL),
    (dict(k_pe=torch.zeros(4, 64, dtype=BF)), SHAPE), (dict(latent=torch.zeros(5, 1, 512, dtype=BF)), SHAPE),
    (dict(kc=torch.zeros(8, 16, 1, 576, dtype=torch.uint8).view(F8), scales=torch.ones(8)), SHAPE),
    (dict(scales=torch.ones(8, 1)), DTYPE), (dict(latent=torch.zeros(5, 512)), DTYPE), (dict(kc=torch.zeros(8, 16, 1, 576)), DTYPE),
    (dict(latent=torch.zeros(5, 256, dtype=BF)), UNSUPPORTED), (dict(k_pe=torch.zeros(5, 128, dtype=BF)), UNSUPPORTED),
    (dict(kc=torch.zeros(8, 16, 2, 576, dtype=BF)), UNSUPPORTED), (dict(kc=torch.zeros(8, 16, 1, 512, dtype=BF)), UNSUPPORTED),
    (dict(cos_sin=torch.zeros(64, 32)), UNSUPPORTED), (dict(cos_sin=torch.zeros(64, 128)), UNSUPPORTED),
    (dict(kc=torch.zeros(8, 16, 1, 576, dtype=torch.uint8).view(F8), scales=torch.ones(8, 1), descale=torch.ones(1)), UNSUPPORTED),
    (dict(latent=torch.zeros(5, 1024, dtype=BF)[:, ::2]), LAYOUT), (dict(k_pe=torch.zeros(5, 68, dtype=BF)[:, 4:]), LAYOUT),
    (dict(kc=torch.zeros(8, 1, 1, 576, dtype=BF).expand(8, 16, 1, 576)), LAYOUT),
]


@pytest.mark.parametrize("i", range(len(MLA_BAD)))
def test_append_mla_refuses(i):
    kw, code = MLA_BAD[i]
    assert call_mla(**kw) == code


def test_calls_without_tokens_are_fine_without_a_gpu():
    """Nothing to store: success before any CUDA call."""
    e = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    assert call_kv(q=e(0, 4, 256), q_out=e(0, 4, 256), k=e(0, 2, 256), v=e(0, 2, 256), cu=torch.zeros(3, dtype=torch.int32)) == 0
    assert call_mla(q=e(0, 4, 64), q_out=e(0, 4, 64), latent=e(0, 512), k_pe=e(0, 64), cu=torch.zeros(3, dtype=torch.int32)) == 0


def test_binding_checks():
    a = kv_args()
    with pytest.raises(ValueError, match="CUDA"):
        va.append_kv(a["k"], a["v"], a["kc"], a["vc"], a["bt"], a["cu"], a["su"])
    with pytest.raises(TypeError):
        va.append_kv(a["k"].half(), a["v"], a["kc"], a["vc"], a["bt"], a["cu"], a["su"])
    with pytest.raises(ValueError, match="positions"):
        va.append_kv(a["k"], a["v"], a["kc"], a["vc"], a["bt"], a["cu"], a["su"], positions=torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError, match="different devices"):
        va.append_kv(a["k"], a["v"].to("meta"), a["kc"], a["vc"], a["bt"], a["cu"], a["su"])
    with pytest.raises(ValueError, match="dimensions"):
        va.append_kv(a["k"][None, None], a["v"], a["kc"], a["vc"], a["bt"], a["cu"], a["su"])


# ---- the oracle itself ------------------------------------------------------------


def test_oracle_rotation_is_a_rotation():
    """Lengths of pairs stay, and a product of two rotated rows depends on the distance alone."""
    rng = np.random.default_rng(0)
    cs = np.asarray(table(64, 32).double())
    q, k = rng.standard_normal(64), rng.standard_normal(64)
    for inter in (False, True):
        dots = [rotated(q, cs, p + 7, inter) @ rotated(k, cs, p, inter) for p in (0, 5, 40)]
        assert np.allclose(dots, dots[0], rtol=0, atol=1e-5)      # the table is in fp32
        y = rotated(k, cs, 3, inter)
        assert np.array_equal(y[32:], k[32:])
        a, b = (slice(0, 32, 2), slice(1, 32, 2)) if inter else (slice(0, 16), slice(16, 32))
        assert np.allclose(y[a] ** 2 + y[b] ** 2, k[a] ** 2 + k[b] ** 2, rtol=1e-6)
        # a quarter turn takes (x1, x2) to (-x2, x1)
        quarter = np.concatenate([np.zeros((1, 16)), np.ones((1, 16))], axis=1)
        z = rotated(k, quarter, 0, inter)
        assert np.array_equal(z[a], -k[b]) and np.array_equal(z[b], k[a])


def test_oracle_scale_rule():
    assert page_scale(448.0) == 1.0 and page_scale(np.nextafter(448.0, 1e9)) == 2.0 and page_scale(224.0) == 0.5
    assert page_scale(0.0) == 2.0 ** -64 and page_scale(math.inf) == 2.0 ** 64 and page_scale(1e-30) == 2.0 ** -64
    for a in (1.0, 3.7, 1e-5, 6e7):
        s = page_scale(a)
        assert math.frexp(s)[0] == 0.5 and a <= 448 * s and a > 448 * s / 2
    assert usable(float("nan")) == 2.0 ** -64 and usable(-3.0) == 2.0 ** -64 and usable(1e30) == 2.0 ** 64


def test_oracle_places_tokens():
    """Token t of L at S - L + t, through the table; older tokens of the first page are kept."""
    rows = np.arange(1.0, 6.0)[:, None, None] * np.ones((5, 1, 4))
    st = append_oracle(rows, np.array([[2, 0], [1, 3]]), [0, 3, 5], [18, 1], 4, before=np.ones((4, 16, 1, 4)),
                       scales=np.full((4, 1), 0.5), limit=448.0)
    assert [(int(p), int(s)) for p, s in np.argwhere(st.written)] == [(0, 0), (0, 1), (1, 0), (2, 15)]
    assert st.value[2, 15, 0, 0] == 1 and st.value[0, 0, 0, 0] == 2 and st.value[0, 1, 0, 0] == 3 and st.value[1, 0, 0, 0] == 5
    assert st.kept[2, :15].all() and st.kept.sum() == 15 and (st.value[2, :15] == 0.5).all()
    assert st.scales[2, 0] == 0.5 and st.scales[0, 0] == page_scale(3.0) and st.scales[3, 0] == 0.5
