"""The page pool's oracle where a row's count cannot be right (CPU)."""
import pytest

from oracle import page_pool as pool


def two_rows(**kw):
    p = dict(table=[[0, 1, -7, -7], [2, 3, -7, -7]], used=[20, 20], count=[2, 2], refs=[1, 1, 1, 1, 0, 0, 0, 0])
    p.update(kw)
    return p


@pytest.mark.parametrize("used,short", [(31, False), (32, False), (33, True), (47, True), (48, True), (49, True)])
def test_reserve_with_fewer_pages_than_tokens(used, short):
    p = two_rows(used=[used, 20])
    status, src, dst, room = pool.reserve(*p.values(), [2, 13])
    assert status == (pool.BAD_TABLE if short else 0)
    assert p["count"][1] == 3 and room[1] == 48 and (src, dst) == ([-1, -1], [-1, -1])
    assert room[0] == 16 * p["count"][0] and p["count"][0] == (2 if short else 3)


@pytest.mark.parametrize("count", [-1, 5, 9])
def test_free_with_a_count_outside_the_row(count):
    p = two_rows(count=[count, 2])
    assert pool.free(*p.values(), [0, 1, 0]) == pool.BAD_TABLE
    assert p["count"] == [count, 0] and p["used"] == [20, 0] and p["refs"][:4] == [1, 1, 0, 0]
