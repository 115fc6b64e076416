"""verify_attn_chunk at the last positions that a block table reaches, 2^31 - 16 of them:
one page stands for all (a table of stride 0), a window and the first tokens are seen."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import decode, gpu
from chunk_util import Chunk, tolerance

pytestmark = pytest.mark.gpu

WIDTH = (2 ** 31 - 1) // 16


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "scaled"])
@pytest.mark.parametrize("S", [16 * WIDTH, 16 * WIDTH - 111, 16 * WIDTH - 112, 16 * WIDTH - 113, 2 ** 30 + 5, 2 ** 31 - 1])
@pytest.mark.parametrize("window,first,splits", [(100, 20, 0), (700, 3, 4), (0, 0, 0)])
def test_last_positions(window, first, splits, S, kind):
    b = Chunk([3], [16], 4, 2, kind, 51)
    table = gpu(b.table[:1, :1]).expand(1, WIDTH)
    used = torch.tensor([S], dtype=torch.int32)
    S = min(S, 16 * WIDTH)                            # (past the table: its width)
    k, v = (b.values(i)[int(b.table[0, 0])] for i in range(2))
    q, want, size = decode(b.q), np.zeros((3, 4, 256)), np.zeros((3, 4, 256))
    for t in range(3):
        i = S - 3 + t
        j = np.concatenate([np.arange(first), np.arange(i - window, i + 1)]) % 16
        for h in range(4):
            s = b.scale * (k[j, h // 2] @ q[t, h])
            p = np.exp(s - s.max())
            want[t, h], size[t, h] = p @ v[j, h // 2] / p.sum(), p @ np.abs(v[j, h // 2]) / p.sum()
    b.used = torch.tensor([window + 1 + first], dtype=torch.int32)   # (the keys that a row sees, for the bound)
    out = va.verify_attn_chunk(gpu(b.q), gpu(b.caches[0]), gpu(b.caches[1]), table, gpu(b.cu), gpu(used), b.scale, k_descale=gpu(b.descales[0]),
                               v_descale=gpu(b.descales[1]), k_scales=gpu(b.scales[0]), v_scales=gpu(b.scales[1]), window_left=window,
                               first_tokens=first, num_splits=splits)
    assert va.last_device_error() == 0
    assert (np.abs(decode(out) - want) <= tolerance(b, want, size)).all()
