"""Vectors of the pool's calls in one place are refused, as are addresses off 4 bytes."""
import ctypes

import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from test_page_pool import LAYOUT, UNSUPPORTED, BF, call, copy, ints
from test_chunk_validation import args as chunk_args


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verify_split_gb300.build import build_library
    build_library()


SHARED, WIDE = ints(4), ints(40)


@pytest.mark.parametrize("which,names", [
    ("reserve", ("new", "src")), ("reserve", ("new", "room")), ("reserve", ("src", "dst")), ("reserve", ("dst", "room")),
    ("reserve", ("su", "new")), ("reserve", ("su", "room")), ("reserve", ("pc", "dst")), ("free", ("su", "pc")), ("fork", ("su", "pc")),
])
def test_one_vector_twice(which, names):
    assert call(which, **{n: SHARED for n in names}) == LAYOUT


@pytest.mark.parametrize("which,kw", [
    ("free", dict(refs=WIDE[:20], a=WIDE[19:22])), ("fork", dict(refs=WIDE[2:22], b=WIDE[:3])), ("fork", dict(pc=WIDE[:4], a=WIDE[3:6])),
    ("reserve", dict(refs=WIDE[:20], room=WIDE[16:20])), ("reserve", dict(src=WIDE[:4], dst=WIDE[3:7])),
])
def test_vectors_that_reach_into_each_other(which, kw):
    assert call(which, **kw) == LAYOUT


def test_rows_too_wide_for_one_launch():
    big = torch.zeros(1, dtype=BF).expand(8, 16, 1 << 16, 256)
    assert copy(k=big, v=None) == UNSUPPORTED


@pytest.mark.parametrize("name", ["bt", "cu", "su"])
def test_chunk_addresses_off_four_bytes(name):
    a = chunk_args()
    d = {n: va.desc(a[n]) for n in ("q", "k", "v", "bt", "cu", "su", "out")}
    d[name].data = d[name].data + 2
    r = {n: ctypes.byref(x) for n, x in d.items()}
    s = va.library().verify_attn_chunk(r["q"], r["k"], r["v"], None, None, r["bt"], r["cu"], r["su"], 1.0, None, None, r["out"], None, 0, None, 0, 0,
                                       None)
    assert s == LAYOUT
