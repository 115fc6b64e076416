"""verify_attn_chunk over its range: caches of tens of thousands of keys, any number of query
heads a KV head, long prompts beside single tokens."""
import pytest

from chunk_util import Chunk, check

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "e4m3", "scaled"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv", [
    ([2, 1], [40000, 70001], 4, 2),
    ([3], [131072], 2, 1),
    ([1, 1, 40, 1], [20001, 5, 9000, 33333], 2, 1),
])
def test_long_caches(q_lens, kv_lens, hq, hkv, kind):
    b = Chunk(q_lens, kv_lens, hq, hkv, kind, 81)
    check(b)
    check(b, window_left=15000, first_tokens=3001)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group,hkv", [(255, 1), (256, 1), (257, 1), (300, 2), (512, 1), (1000, 1)])
def test_many_heads(group, hkv, kind):
    b = Chunk([2, 0, 3], [150, 20, 3], group * hkv, hkv, kind, 82, tail=1)
    check(b, sinks=True)
    check(b, sinks=True, window_left=40, first_tokens=2, run_kw=dict(num_splits=9))


@pytest.mark.parametrize("kind", KINDS)
def test_prompts_beside_single_tokens(kind):
    q = [1] * 14 + [1700] + [1] * 15 + [300, 0, 4]
    kv = [2000 + 251 * i for i in range(14)] + [1700] + [100 + 613 * i for i in range(15)] + [2100, 9, 4096]
    b = Chunk(q, kv, 2, 1, kind, 83)
    check(b)
    check(b, window_left=511, first_tokens=4, sinks=True)
