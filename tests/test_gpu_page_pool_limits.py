"""The page pool's calls where counts do not fit: more pages wanted than 31 bits hold,
counts that belong to no row, rows of a cache as wide as a launch takes."""
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from test_gpu_page_pool import Both

pytestmark = pytest.mark.gpu
I = torch.int32


def test_more_pages_wanted_than_31_bits():
    """Sequences behind the sum that passes 2^31 get nothing either, and it is reported."""
    seqs, width, pages = 8192, 262400, 64
    table = torch.empty(seqs, width, dtype=I, device="cuda")     # 8.6 GB; no row holds a page
    used, count = (torch.zeros(seqs, dtype=I, device="cuda") for _ in range(2))
    refs, status = torch.zeros(pages, dtype=I, device="cuda"), torch.zeros(1, dtype=I, device="cuda")
    add = torch.full((seqs,), 16 * width, dtype=I, device="cuda")
    add[-3] = 0
    src, dst, room = va.reserve_pages(table, used, count, refs, add, status=status)
    torch.cuda.synchronize()
    assert int(status) == va.PG_NO_PAGES
    assert int(count.abs().max()) == 0 and int(refs.abs().max()) == 0 and int(room.abs().max()) == 0
    assert (src == -1).all() and (dst == -1).all()
    add.zero_()
    add[0], add[-1] = 16, 40                                     # (and the pool is as it was)
    va.reserve_pages(table, used, count, refs, add, status=status)
    torch.cuda.synchronize()
    assert count.nonzero().flatten().tolist() == [0, seqs - 1] and table[0, 0] == 0 and table[-1, :3].tolist() == [1, 2, 3]


@pytest.mark.parametrize("dtype,heads", [(torch.bfloat16, 65535), (torch.float8_e4m3fn, 131070)])
def test_pages_as_wide_as_a_launch_takes(dtype, heads):
    """Token rows of 65,535 * 512 bytes: the last CTA of the launch has the page's end."""
    k = torch.empty(3, 16, heads, 256, dtype=dtype, device="cuda")
    bits = k.view(torch.uint8).view(3, -1)
    bits[0] = torch.arange(bits.shape[1], device="cuda") % 251
    bits[1:] = 253
    va.copy_pages(k, None, torch.tensor([0], dtype=I, device="cuda"), torch.tensor([2], dtype=I, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(bits[0], bits[2]) and bool((bits[1] == 253).all())
