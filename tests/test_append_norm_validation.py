"""Refusals of append_kv_norm: status codes from the host checks, before any launch."""
import ctypes

import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import descriptors, rope_of
from test_append_validation import kv_args

NULL, SHAPE, DTYPE, UNSUPPORTED, LAYOUT = 1, 2, 3, 4, 7
BF = torch.bfloat16
W = torch.ones(256, dtype=BF)


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verify_split_gb300.build import build_library
    build_library()


def call(qw=None, kw=None, eps=1e-6, offset=0.0, norm=True, **over):
    a = kv_args(**over)
    r = descriptors(a["q"], a["k"], a["v"], a["bt"], a["cu"], a["su"], a["kd"], a["vd"], a["ks"], a["vs"], a["q_out"], a["kc"], a["vc"])
    n = va.VaNorm(*descriptors(qw, kw), eps, offset)
    return va.library().verify_attn_append_kv_norm(*r[:6], ctypes.pointer(n) if norm else None,
                                                   rope_of(a["cos_sin"], a["positions"], a["interleaved"]), *r[6:], None)


BAD = [
    (dict(qw=torch.ones(255, dtype=BF)), SHAPE), (dict(kw=torch.ones(2, 128, dtype=BF)), SHAPE),
    (dict(qw=torch.ones(256, dtype=torch.int32)), DTYPE), (dict(kw=torch.zeros(256, dtype=torch.uint8).view(torch.float8_e4m3fn)), DTYPE),
    (dict(qw=torch.ones(512, dtype=BF)[::2]), LAYOUT), (dict(kw=torch.ones(260, dtype=BF)[4:]), LAYOUT),
    (dict(qw=W, eps=-1e-6), UNSUPPORTED), (dict(qw=W, eps=float("nan")), UNSUPPORTED), (dict(kw=W, eps=float("inf")), UNSUPPORTED),
    (dict(kw=W, offset=float("inf")), UNSUPPORTED), (dict(kw=W, offset=float("nan")), UNSUPPORTED),
    (dict(qw=W, q=None, q_out=None), NULL), (dict(qw=W, q_out=None), NULL),
    (dict(kw=W, cos_sin=None), NULL),                        # queries with nothing to do
    (dict(cos_sin=None), NULL), (dict(norm=False, cos_sin=None), NULL),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_refuses(i):
    kw, code = BAD[i]
    assert call(**kw) == code


def test_nothing_to_store_is_fine_without_a_gpu():
    e = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    none = dict(q=e(0, 4, 256), q_out=e(0, 4, 256), k=e(0, 2, 256), v=e(0, 2, 256), cu=torch.zeros(3, dtype=torch.int32))
    assert call(qw=W, kw=W, **none) == 0
    assert call(qw=W, cos_sin=None, **none) == 0             # norms without a rotation
    assert call(norm=False, **none) == 0


def test_binding_checks():
    a = kv_args()
    with pytest.raises(ValueError, match="CUDA"):
        va.append_kv(a["k"], a["v"], a["kc"], a["vc"], a["bt"], a["cu"], a["su"], k_norm=W)
    with pytest.raises(TypeError):
        va.append_kv(a["k"], a["v"], a["kc"], a["vc"], a["bt"], a["cu"], a["su"], k_norm=W.half())
    with pytest.raises(ValueError, match="different devices"):
        va.append_kv(a["k"], a["v"], a["kc"], a["vc"], a["bt"], a["cu"], a["su"], k_norm=W.to("meta"))
