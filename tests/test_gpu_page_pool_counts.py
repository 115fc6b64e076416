"""Rows of the page pool whose counts cannot be right are reported and left as they are."""
import pytest

import speculative_decoding_verify_split_gb300 as va
from test_gpu_page_pool import Both

pytestmark = pytest.mark.gpu


def two_rows():
    b = Both(2, 4, 16)
    *_, room = b.reserve([20, 20])
    b.write([20, 20], room)
    return b


@pytest.mark.parametrize("used,short", [(32, False), (33, True), (40, True), (48, True), (49, True), (60, True)])
def test_reserve_with_fewer_pages_than_tokens(used, short):
    b = two_rows()
    b.set(used=[used, 20])
    *_, room = b.reserve([4, 30])
    assert b.bits == (va.PG_BAD_TABLE if short else 0)
    assert b.count.tolist() == [2 if short else 3, 4] and room == [32 if short else 48, 64]


@pytest.mark.parametrize("count", [-1, -(1 << 31), 5, 9, (1 << 31) - 1])
@pytest.mark.parametrize("seqs", [[0, 1], [1, 0, 0], [0] * 40 + [1]])
def test_free_with_a_count_outside_the_row(seqs, count):
    b = two_rows()
    b.set(count=[count, 2])
    b.free(seqs)
    assert b.bits == va.PG_BAD_TABLE
    assert b.count.tolist() == [count, 0] and b.used.tolist() == [20, 0] and b.refs.tolist()[:5] == [1, 1, 0, 0, 0]
    b.set(count=[2, 0])
    b.free(seqs)                                     # put right, it goes back as any other
    assert b.refs.tolist() == [0] * 16
