"""verify_attn_chunk over e4m3 caches where one key, of value 0, outweighs all others: what is
left of a row are their weights, in the documented steps."""
import math

import numpy as np
import pytest

from append_util import decode
from chunk_util import Chunk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("kind", ["e4m3", "scaled"])
@pytest.mark.parametrize("at", [0, 77, 500, 694])
@pytest.mark.parametrize("above", [8, 20, 24, 28, 34])
def test_one_key_above_the_others(above, at, kind, splits):
    b = Chunk([5], [700], 2, 1, kind, 71)
    b.q.zero_()
    b.q[..., 0] = 1.0
    b.scale = math.log(2) * above / 32                # that many log2 units for a product of 32
    if kind == "scaled":
        for s in b.scales:
            s.fill_(1.0)
    else:
        for s in b.descales:
            s.fill_(1.0)
    for p in range(44):
        b.caches[0][int(b.table[0, p]), :, :, 0] = 0.0
    page, slot = int(b.table[0, at // 16]), at % 16
    b.caches[0][page, slot, 0, 0] = 32.0
    b.caches[1][page, slot] = 0.0
    want, size = b.expect()
    out = decode(b.run(num_splits=splits))
    # the output's rounding and the weights', 2^-11 of each or half a step of 2^-31 of the
    # largest (whose p_j is 1 / l, at most 1); exponents and sums in fp32 as in `tolerance`
    v = np.abs(b.values(1))[b.table[0].numpy(), :, 0].reshape(-1, 256)
    steps = np.stack([2.0 ** -32 * v[:696 + t].sum(axis=0) for t in range(5)])[:, None]
    logit = 256 * 2.0 ** -24 * above * math.log(2) + 2.0 ** -21 * 1.45 * above * math.log(2) + 2.0 ** -21
    assert (np.abs(out - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * logit) * size + steps).all()
    if above <= 24:                                   # a step is 2^-7 of such a weight: the row keeps its direction
        err = np.sqrt(((out - want) ** 2).sum(axis=2) / (want ** 2).sum(axis=2))
        assert (err <= 2.0 ** -7).all()
