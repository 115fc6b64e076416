"""copy_pages: the widest token rows that one launch takes, and the first that it refuses (CPU)."""
import pytest
import torch

from test_page_pool import BF, F8, LAYOUT, UNSUPPORTED, copy


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verify_split_gb300.build import build_library
    build_library()


def wide(dtype, heads, dim):
    return torch.zeros(1, dtype=dtype).expand(8, 16, heads, dim)


# a CTA moves 8 KB of a page, 65,535 CTAs a page: rows of 65,535 * 512 bytes
@pytest.mark.parametrize("dtype,dim,heads", [(BF, 256, 65535), (BF, 16776960, 1), (F8, 512, 65535), (F8, 33553920, 1)])
def test_widest_rows(dtype, dim, heads):
    assert copy(k=wide(dtype, heads, dim), v=None) == LAYOUT     # (the next check: these lie on top of each other)


@pytest.mark.parametrize("dtype,dim,heads", [(BF, 256, 65536), (BF, 16776968, 1), (BF, (1 << 24) - 8, 1), (F8, 512, 65536), (F8, 33553936, 1),
                                             (F8, (1 << 25) - 16, 1), (BF, 1 << 40, 1), (F8, 16, 1 << 50)])
def test_rows_too_wide(dtype, dim, heads):
    assert copy(k=wide(dtype, heads, dim), v=None) == UNSUPPORTED
