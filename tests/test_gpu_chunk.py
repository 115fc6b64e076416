"""verify_attn_chunk against the fp64 oracle: row tiles and key tiles that end
anywhere, every cache type, windows with first tokens, shares of the work."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import decode, gpu
from chunk_util import Chunk, check

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "scaled"]


@pytest.mark.parametrize("kind", KINDS)
def test_one_token(kind):
    check(Chunk([1], [1], 1, 1, kind, 0))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv", [
    ([128], [128], 1, 1),            # one CTA's rows, one key tile
    ([256], [256], 1, 1),            # a pair's rows
    ([257], [300], 1, 1),            # one row more
    ([16], [1024], 16, 1),
    ([17, 40, 1], [200, 391, 129], 16, 1),
    ([3, 0, 70, 5], [3, 50, 70, 2000], 8, 2),
    ([33], [160], 3, 1),             # heads that do not divide a row tile
    ([90], [91], 5, 1),
    ([20, 31], [31, 47], 20, 4),
    ([5, 7], [3, 7], 4, 1),          # tokens before position 0 see nothing
    ([4], [0], 2, 1),                # nothing cached at all
])
def test_shapes(q_lens, kv_lens, hq, hkv, kind):
    check(Chunk(q_lens, kv_lens, hq, hkv, kind, sum(kv_lens) + hq, tail=2))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [0, 1, 2, 5, 64])
def test_shares(splits, kind):
    check(Chunk([20, 1, 33], [900, 700, 33], 8, 1, kind, 11), run_kw=dict(num_splits=splits))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,first", [(0, 0), (0, 1), (5, 4), (63, 0), (127, 130), (200, 16), (500, 3), (1 << 30, 7), (31, 2000)])
def test_windows_and_first_tokens(window, first, kind):
    check(Chunk([40, 1, 7], [700, 513, 7], 4, 1, kind, window % 97 + first), window_left=window, first_tokens=first)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [0, 1, 7])
def test_softcap_and_sinks(kind, splits):
    b = Chunk([20, 2], [300, 400], 8, 2, kind, 3, spread=4.0)
    check(b, sinks=True, softcap=15.0, run_kw=dict(num_splits=splits))
    check(b, sinks=True, run_kw=dict(num_splits=splits))
    check(b, sinks=True, softcap=8.0, window_left=100, first_tokens=4, run_kw=dict(num_splits=splits))
