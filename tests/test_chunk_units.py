"""verify_attn_chunk: the split's units fit 63 bits whatever the prefix sums say (every
sequence may then claim all rows of q), or the call is refused (CPU)."""
import ctypes

import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import descriptors
from test_chunk_validation import BF, I, UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verify_split_gb300.build import build_library
    build_library()


@pytest.mark.parametrize("seqs,tokens,width,refused", [
    (1 << 14, 1 << 18, (1 << 27) - 1, True), (1 << 12, 1 << 16, (1 << 27) - 1, False), (1 << 14, 1 << 18, 1 << 16, False),
    (1, 1 << 26, (1 << 27) - 1, False), (1 << 20, 1 << 20, 64, False),
])
def test_units_of_broken_prefix_sums(seqs, tokens, width, refused):
    rows = torch.zeros(8, 256, dtype=BF).as_strided((tokens, 16, 256), (0, 0, 1))
    q, out = va.desc(rows), va.desc(rows)
    for i, n in enumerate((16 * 256, 256, 1)):
        out.stride[i] = n                    # (described, not there: without a GPU no call gets further)
    k = torch.zeros(8, 16, 1, 256, dtype=BF)
    table = torch.zeros(1, 1, dtype=I).expand(seqs, width)
    r = descriptors(k, torch.ones(8, 16, 1, 256, dtype=BF), table, torch.zeros(seqs + 1, dtype=I), torch.zeros(seqs, dtype=I))
    if torch.cuda.is_available() and not refused:
        pytest.skip("would run")
    s = va.library().verify_attn_chunk(ctypes.byref(q), r[0], r[1], None, None, *r[2:], 1.0, None, None, ctypes.byref(out), None, 0, None, 0, 0, None)
    assert (s == UNSUPPORTED) == refused
