"""verify_attn_chunk where an item's last row lies inside a warp's 32: whole items and
items that pairs share."""
import pytest

from chunk_util import Chunk, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "scaled"])
@pytest.mark.parametrize("rows", [1, 31, 32, 33, 63, 65, 95, 97, 127, 129, 161, 225, 255])
def test_rows_that_end_inside_a_warp(rows, kind):
    b = Chunk([rows], [rows + 400], 1, 1, kind, rows, tail=1)
    check(b, run_kw=dict(num_splits=1))              # written from the item itself
    check(b, run_kw=dict(num_splits=3))              # joined from partials


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "scaled"])
def test_variants_over_such_rows(kind):
    b = Chunk([11, 1, 27], [300, 150, 27], 7, 1, kind, 42)
    check(b, sinks=True, softcap=9.0, window_left=90, first_tokens=3)
    check(b, sinks=True, softcap=9.0, window_left=90, first_tokens=3, run_kw=dict(num_splits=4))
