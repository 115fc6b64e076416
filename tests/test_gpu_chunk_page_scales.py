"""verify_attn_chunk over pages whose V scales lie far apart: the normaliser counts the keys
of the smaller ones, up to the documented 2^-126 of the row's largest weight times scale."""
import numpy as np
import pytest
import torch

from append_util import decode
from chunk_util import Chunk, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("apart", [20, 60, 100, 124])
@pytest.mark.parametrize("large", [[0], [1], [20], [0, 3, 9, 17, 20], list(range(1, 21))])
def test_scales_far_apart(large, apart, splits):
    """Equal logits, so a key's weight is one of the row's count whatever its page's scale."""
    b = Chunk([3, 40], [330, 330], 4, 1, "scaled", 61)
    b.q.zero_()
    scale = torch.full((b.pages, 1), 2.0 ** -(apart // 2))
    for s in range(2):
        for p in large:
            scale[int(b.table[s, p])] = 2.0 ** (apart - apart // 2)
    b.scales[1] = scale
    want, size = b.expect()
    out = decode(b.run(num_splits=splits))
    assert np.isfinite(out).all()
    assert (np.abs(out - want) <= tolerance(b, want, size)).all()


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("apart", [30, 110])
def test_a_page_of_zeros_with_a_large_scale(apart, splits):
    """The page with the large scale holds values of 0: what is left are the others, in the
    documented steps of their weight times scale."""
    b = Chunk([5], [200], 2, 1, "scaled", 62)
    b.q.zero_()
    b.scales[1] = torch.full((b.pages, 1), 2.0 ** -40)
    page = int(b.table[0, 4])
    b.scales[1][page] = 2.0 ** (apart - 40)
    b.caches[1][page] = 0.0
    want, size = b.expect()
    out = decode(b.run(num_splits=splits))
    # a step of 2^-31 of the largest weight times scale, half of it a key
    seen = np.arange(196, 201)[:, None, None]
    steps = 2.0 ** -32 * 2.0 ** (apart - 40) * 448
    assert (np.abs(out - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -19) * size + steps * seen / seen).all()
    assert (np.abs(out) <= 2.0 ** -40 * 448).all()
