"""The records of verify_attn_chunk's split, as the call leaves them in the workspace for
its merge: every share starts in the item that holds its first unit, and nothing that the
main kernel does at the same time reaches the record. Calls of few and short items leave
nothing to join."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import gpu
from chunk_util import Chunk

pytestmark = pytest.mark.gpu

RECORD = np.dtype([("off", "<i8"), ("total", "<i8"), ("b", "<i4"), ("h", "<i4"), ("m", "<i4"), ("used", "<i4")])
ROWS, KEYS, ITEM = 256, 128, 5  # an item's rows, a tile's keys, an item's cost beside its tiles in tiles
WHOLE = 18                      # .. and what an item that a pair has to itself costs at most


def items(b, window=-1, first=0):
    """[(first unit, behind the last one, sequence, head, row tile)] in the split's order."""
    group, at, out = b.hq // b.hkv, 0, []
    cap = (window + 2 + first) * group + ROWS if window >= 0 else 1 << 60
    for s in range(len(b.used)):
        L, S = int(b.cu[s + 1] - b.cu[s]), int(b.used[s])
        for h in range(b.hkv):
            for m in range(-(-L * group // ROWS)):
                cost = min(max(0, (S - L) * group + ROWS * (m + 1)), cap) + ITEM * KEYS * group
                out.append((at, at + cost, s, h, m))
                at += cost
    return out


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "scaled"])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,kw", [
    ([25, 21], [461, 320], 16, 1, {}),               # few and short: a pair an item
    ([25, 21], [461, 320], 16, 1, dict(num_splits=7)),
    ([25, 21], [461, 1600], 16, 1, {}),              # .. one of 13 tiles
    ([25, 21], [461, 1700], 16, 1, {}),              # .. one of 14
    ([250] * 5, [300] * 5, 16, 1, {}),               # more items than pairs
    ([700, 1, 33], [700, 2000, 900], 8, 2, {}),
    ([1] * 40, [600 + 9 * i for i in range(40)], 16, 2, dict(window_left=255, first_tokens=4)),
    ([40, 3, 0, 200], [4000, 3, 50, 1200], 3, 1, dict(num_splits=76)),
])
def test_shares_start_where_their_records_say(q_lens, kv_lens, hq, hkv, kw, kind):
    b = Chunk(q_lens, kv_lens, hq, hkv, kind, 41)
    want = items(b, kw.get("window_left", -1), kw.get("first_tokens", 0))
    total = want[-1][1]
    ws = torch.zeros(va.chunk_workspace_size(), dtype=torch.uint8, device="cuda")
    at = (-ws.data_ptr()) % 256 + 256                 # (behind the status word)
    args = b.args()
    more = dict(k_descale=gpu(b.descales[0]), v_descale=gpu(b.descales[1]), k_scales=gpu(b.scales[0]), v_scales=gpu(b.scales[1]))
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    records, eager = ws[at:at + pairs * RECORD.itemsize], None
    for _ in range(30):
        records.fill_(0xEE)
        out = va.verify_attn_chunk(*args, b.scale, workspace=ws, **more, **kw)
        rec = records.cpu().numpy().view(RECORD)
        used = int(rec["used"][0])
        if not kw.get("num_splits") and len(want) <= pairs and max(z - a for a, z, *_ in want) <= WHOLE * KEYS * (hq // hkv):
            assert used == 0
        else:
            assert 0 < used <= pairs
        share = -(-total // max(used, 1))
        for c in range(used):
            i0, i1, s, h, m = next(x for x in want if x[0] <= c * share < x[1])
            assert tuple(rec[c]) == (i0, total, s, h, m, used)
        eager = out if eager is None else eager
        assert torch.equal(out, eager)
    assert va.workspace_status(ws) == 0
