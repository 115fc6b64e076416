"""The page-scaled attention's oracle pinned to the plain ones, and the host
checks of verify_attn_scaled and verify_attn_mla_scaled (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import decode, descriptors
from oracle.attention_fp64 import oracle_from_torch
from oracle.mla_fp64 import mla_oracle_from_torch
from oracle.page_scaled_fp64 import page_scaled_oracle, read_scales
from speculative_decoding_verify_split_gb300.workloads import make_mla_workload, make_workload

NULL, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE, LAYOUT = 1, 2, 3, 4, 5, 7
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verify_split_gb300.build import build_library
    build_library()


def oracle_of(w, ks, vs, **kw):
    return page_scaled_oracle(decode(w.q), np.nan_to_num(decode(w.k_cache)), np.nan_to_num(decode(w.v_cache)), ks, vs,
                              w.block_table.numpy(), w.cu_seqlens_q.numpy(), w.seqused_k.numpy(), w.softmax_scale, **kw)


@pytest.mark.parametrize("kw", [{}, dict(window_left=40), dict(softcap=5.0), dict(sinks=np.linspace(-2, 2, 8))])
def test_oracle_with_equal_scales_is_the_plain_one(kw):
    """One scale everywhere is a descale."""
    w = make_workload([4, 2, 3, 1], [100, 33, 2, 16], 8, 2, "fp8_e4m3", seed=3, k_descale=0.5, v_descale=4.0)
    n = w.k_cache.shape[0]
    got, tol = oracle_of(w, np.full((n, 2), 0.5), np.full((n, 2), 4.0), **kw)
    assert np.allclose(got, oracle_from_torch(w, **kw), rtol=0, atol=1e-12)
    assert (tol[np.abs(got) > 0] > 0).all()


def test_oracle_with_page_scales_is_the_plain_one_on_scaled_codes():
    """Powers of two moved from the scales into codes that can hold them."""
    w = make_workload([3, 2], [90, 47], 4, 2, "fp8_e4m3", seed=4)
    n = w.k_cache.shape[0]
    g = torch.Generator().manual_seed(1)
    e = [torch.randint(0, 4, (n, 2), generator=g).float() for _ in range(2)]
    got, _ = oracle_of(w, torch.exp2(e[0]).numpy(), torch.exp2(e[1]).numpy())
    for c, x in ((w.k_cache, e[0]), (w.v_cache, e[1])):
        y = c.float() * torch.exp2(x)[:, None, :, None]
        assert torch.equal(torch.nan_to_num(y.to(F8).float()), torch.nan_to_num(y))
        c.view(torch.uint8).copy_(y.to(F8).view(torch.uint8))
    assert np.allclose(got, oracle_from_torch(w), rtol=0, atol=1e-12)


def test_oracle_on_a_latent_cache():
    w = make_mla_workload([2, 3], [70, 20], 4, "fp8_e4m3", seed=5, k_descale=0.25, v_descale=0.25)
    n = w.kv_cache.shape[0]
    c = np.nan_to_num(decode(w.kv_cache))
    got, _ = page_scaled_oracle(decode(w.q), c, c[..., :512], np.full((n, 1), 0.25), np.full((n, 1), 0.25), w.block_table.numpy(),
                                w.cu_seqlens_q.numpy(), w.seqused_k.numpy(), w.softmax_scale)
    assert np.allclose(got, mla_oracle_from_torch(w), rtol=0, atol=1e-12)


def test_oracle_sees_one_page_scale():
    """The scale of one page matters to the rows that see it, and to no other."""
    w = make_workload([1, 1], [40, 40], 2, 1, "fp8_e4m3", seed=6)
    n = w.k_cache.shape[0]
    base, _ = oracle_of(w, np.ones((n, 1)), np.ones((n, 1)))
    for which in range(2):
        s = [np.ones((n, 1)), np.ones((n, 1))]
        s[which][int(w.block_table[0, 1])] = 3.0
        got, _ = oracle_of(w, *s)
        assert not np.allclose(got[0], base[0]) and np.array_equal(got[1], base[1])
    assert np.array_equal(read_scales(np.array([np.nan, -1, 0, np.inf])), [2.0 ** -64] * 3 + [2.0 ** 64])


def args(**kw):
    f8 = lambda *s: torch.zeros(*s, dtype=torch.uint8).view(F8)  # noqa: E731
    a = dict(q=torch.zeros(5, 4, 256, dtype=BF), kc=f8(8, 16, 2, 256), vc=f8(8, 16, 2, 256), ks=torch.ones(8, 2), vs=torch.ones(8, 2),
             bt=torch.zeros(2, 3, dtype=torch.int32), cu=torch.tensor([0, 2, 5], dtype=torch.int32),
             su=torch.tensor([4, 9], dtype=torch.int32), mq=3, mk=48, out=torch.zeros(5, 4, 256, dtype=BF), sinks=None, win=-1, cap=0.0,
             ws=None, n=0, splits=0)
    a.update(kw)
    return a


def call(**kw):
    a = args(**kw)
    r = descriptors(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["cu"], a["su"], a["out"], a["sinks"])
    opts = ctypes.pointer(va.VaOptions(a["win"], a["cap"], r[9]))
    return va.library().verify_attn_scaled(*r[:8], a["mq"], a["mk"], 0.1, r[8], opts, a["ws"], a["n"], a["splits"], None, None)


BAD = [
    (dict(q=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(ks=None), NULL), (dict(vs=None), NULL), (dict(bt=None), NULL),
    (dict(out=None), NULL),
    (dict(ks=torch.ones(7, 2)), SHAPE), (dict(vs=torch.ones(8, 1)), SHAPE), (dict(ks=torch.ones(16)), SHAPE),
    (dict(mk=64), SHAPE), (dict(sinks=torch.zeros(3)), SHAPE),
    (dict(ks=torch.ones(8, 2, dtype=BF)), DTYPE), (dict(vs=torch.ones(8, 2, dtype=torch.int32)), DTYPE),
    (dict(kc=torch.zeros(8, 16, 2, 256, dtype=BF), vc=torch.zeros(8, 16, 2, 256, dtype=BF)), DTYPE),
    (dict(mq=33), UNSUPPORTED), (dict(win=-2), UNSUPPORTED), (dict(cap=-1.0), UNSUPPORTED), (dict(splits=-1), UNSUPPORTED),
    (dict(ks=torch.ones(1, 2).expand(8, 2)), LAYOUT), (dict(vs=torch.ones(8, 1).expand(8, 2)), LAYOUT),
    (dict(q=torch.zeros(5, 4, 260, dtype=BF)[..., 2:258]), LAYOUT),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_scaled_refuses(i):
    kw, code = BAD[i]
    assert call(**kw) == code


def call_mla(**kw):
    a = dict(q=torch.zeros(5, 4, 576, dtype=BF), kc=torch.zeros(8, 16, 1, 576, dtype=torch.uint8).view(F8), s=torch.ones(8, 1),
             bt=torch.zeros(2, 3, dtype=torch.int32), cu=torch.tensor([0, 2, 5], dtype=torch.int32),
             su=torch.tensor([4, 9], dtype=torch.int32), mq=3, mk=48, out=torch.zeros(5, 4, 512, dtype=BF), splits=0)
    a.update(kw)
    r = descriptors(a["q"], a["kc"], a["s"], a["bt"], a["cu"], a["su"], a["out"])
    return va.library().verify_attn_mla_scaled(*r[:6], a["mq"], a["mk"], 0.1, r[6], None, 0, a["splits"], None, None)


MLA_BAD = [
    (dict(s=None), NULL), (dict(kc=None), NULL), (dict(s=torch.ones(8)), SHAPE), (dict(s=torch.ones(8, 2)), SHAPE), (dict(s=torch.ones(9, 1)), SHAPE),
    (dict(s=torch.ones(8, 1, dtype=BF)), DTYPE), (dict(kc=torch.zeros(8, 16, 1, 576, dtype=BF)), DTYPE),
    (dict(q=torch.zeros(5, 4, 512, dtype=BF)), UNSUPPORTED), (dict(mq=17), UNSUPPORTED), (dict(splits=-1), UNSUPPORTED),
    (dict(s=torch.ones(1, 1).expand(8, 1)), LAYOUT),
]


@pytest.mark.parametrize("i", range(len(MLA_BAD)))
def test_mla_scaled_refuses(i):
    kw, code = MLA_BAD[i]
    assert call_mla(**kw) == code


def test_bindings_refuse_host_tensors():
    a = args()
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        va.verify_attn_scaled(a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["cu"], a["su"], 3, 48, 0.1)
    with pytest.raises(ValueError, match="different devices"):
        va.verify_attn_scaled(a["q"], a["kc"], a["vc"], a["ks"].to("meta"), a["vs"], a["bt"], a["cu"], a["su"], 3, 48, 0.1)
