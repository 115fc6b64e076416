"""The page pool on the CPU: refusals of its calls before any launch, and the
oracle against the rules that a pool keeps."""
import random

import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import descriptors
from oracle import page_pool as pool

NULL, SHAPE, DTYPE, UNSUPPORTED, LAYOUT = 1, 2, 3, 4, 7
BF, F8, I = torch.bfloat16, torch.float8_e4m3fn, torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    from speculative_decoding_verify_split_gb300.build import build_library
    build_library()


def ints(*shape):
    return torch.zeros(*shape, dtype=I)


def pool_args(**kw):
    a = dict(bt=ints(4, 6), su=ints(4), pc=ints(4), refs=ints(20), a=ints(3), b=ints(3), new=ints(4), src=ints(4), dst=ints(4), room=ints(4))
    a.update(kw)
    return a


def call(which, **kw):
    a = pool_args(**kw)
    base = descriptors(a["bt"], a["su"], a["pc"], a["refs"])
    L = va.library()
    if which == "free":
        return L.verify_attn_free_pages(*base, *descriptors(a["a"]), None, None)
    if which == "fork":
        return L.verify_attn_fork_pages(*base, *descriptors(a["a"], a["b"]), None, None)
    return L.verify_attn_reserve_pages(*base, *descriptors(a["new"], a["src"], a["dst"], a["room"]), None, None)


POOL_BAD = [
    (dict(bt=None), NULL), (dict(su=None), NULL), (dict(pc=None), NULL), (dict(refs=None), NULL),
    (dict(bt=ints(24)), SHAPE), (dict(su=ints(3)), SHAPE), (dict(pc=ints(5)), SHAPE), (dict(refs=ints(4, 5)), SHAPE),
    (dict(bt=torch.zeros(4, 6)), DTYPE), (dict(su=torch.zeros(4)), DTYPE), (dict(pc=torch.zeros(4)), DTYPE), (dict(refs=torch.zeros(20)), DTYPE),
    (dict(su=ints(8)[::2]), LAYOUT), (dict(pc=ints(8)[::2]), LAYOUT), (dict(refs=ints(40)[::2]), LAYOUT),
    (dict(bt=ints(1, 6).expand(4, 6)), LAYOUT), (dict(bt=ints(4, 1).expand(4, 6)), LAYOUT),
]


@pytest.mark.parametrize("which", ["free", "fork", "reserve"])
@pytest.mark.parametrize("i", range(len(POOL_BAD)))
def test_pool_refuses(which, i):
    kw, code = POOL_BAD[i]
    assert call(which, **kw) == code


@pytest.mark.parametrize("which,kw,code", [
    ("free", dict(a=None), NULL), ("free", dict(a=ints(3, 1)), SHAPE), ("free", dict(a=torch.zeros(3)), DTYPE), ("free", dict(a=ints(6)[::2]), LAYOUT),
    ("fork", dict(a=None), NULL), ("fork", dict(b=None), NULL), ("fork", dict(b=ints(2)), SHAPE), ("fork", dict(b=torch.zeros(3)), DTYPE),
    ("fork", dict(b=ints(6)[::2]), LAYOUT),
    ("reserve", dict(new=None), NULL), ("reserve", dict(src=None), NULL), ("reserve", dict(dst=None), NULL), ("reserve", dict(room=None), NULL),
    ("reserve", dict(new=ints(3)), SHAPE), ("reserve", dict(room=ints(5)), SHAPE), ("reserve", dict(src=torch.zeros(4)), DTYPE),
    ("reserve", dict(dst=ints(8)[::2]), LAYOUT),
    ("reserve", dict(bt=ints(8193, 1), su=ints(8193), pc=ints(8193), new=ints(8193), src=ints(8193), dst=ints(8193), room=ints(8193)), UNSUPPORTED),
    ("reserve", dict(refs=ints((1 << 22) + 1)), UNSUPPORTED),
    ("free", dict(a=ints(0)), 0), ("fork", dict(a=ints(0), b=ints(0)), 0),
    ("reserve", dict(bt=ints(0, 6), su=ints(0), pc=ints(0), new=ints(0), src=ints(0), dst=ints(0), room=ints(0)), 0),
])
def test_lists_refuse(which, kw, code):
    assert call(which, **kw) == code


def copy(**kw):
    a = dict(k=torch.zeros(8, 16, 2, 256, dtype=BF), v=torch.zeros(8, 16, 2, 256, dtype=BF), ks=None, vs=None, src=ints(3), dst=ints(3))
    a.update(kw)
    return va.library().verify_attn_copy_pages(*descriptors(a["k"], a["v"], a["ks"], a["vs"], a["src"], a["dst"]), None)


E = [torch.zeros(8, 16, 2, 256, dtype=torch.uint8).view(F8) for _ in range(2)]
S = torch.ones(8, 2)
SAME = torch.zeros(8, 16, 2, 256, dtype=BF)
COPY_BAD = [
    (dict(k=None), NULL), (dict(src=None), NULL), (dict(dst=None), NULL), (dict(k=E[0], v=E[1], ks=S), NULL), (dict(k=E[0], v=E[1], vs=S), NULL),
    (dict(k=E[0], v=None, vs=S), NULL),
    (dict(v=torch.zeros(7, 16, 2, 256, dtype=BF)), SHAPE), (dict(k=torch.zeros(8, 16, 512, dtype=BF)), SHAPE), (dict(dst=ints(4)), SHAPE),
    (dict(k=E[0], v=E[1], ks=torch.ones(7, 2), vs=S.clone()), SHAPE),
    (dict(k=torch.zeros(8, 16, 2, 256)), DTYPE), (dict(v=E[0]), DTYPE), (dict(ks=S, vs=S.clone()), DTYPE), (dict(src=torch.zeros(3)), DTYPE),
    (dict(k=E[0], v=E[1], ks=S.to(BF), vs=S.clone()), DTYPE),
    (dict(k=torch.zeros(8, 32, 2, 256, dtype=BF)), UNSUPPORTED), (dict(k=torch.zeros(8, 16, 2, 250, dtype=BF)), UNSUPPORTED),
    (dict(k=torch.zeros(1, 16, 2, 256, dtype=BF).expand(8, 16, 2, 256)), LAYOUT), (dict(k=SAME, v=SAME), LAYOUT),
    (dict(k=torch.zeros(8, 16, 2, 260, dtype=BF)[..., 4:]), LAYOUT), (dict(src=ints(6)[::2]), LAYOUT),
    (dict(k=E[0], v=E[1], ks=S, vs=S), LAYOUT), (dict(k=E[0], v=E[1], ks=torch.ones(1, 2).expand(8, 2), vs=S), LAYOUT),
    (dict(src=ints(0), dst=ints(0)), 0), (dict(k=torch.zeros(0, 16, 2, 256, dtype=BF), v=torch.zeros(0, 16, 2, 256, dtype=BF)), 0),
]


@pytest.mark.parametrize("i", range(len(COPY_BAD)))
def test_copy_refuses(i):
    kw, code = COPY_BAD[i]
    assert copy(**kw) == code


def test_binding_checks():
    a = pool_args()
    with pytest.raises(ValueError, match="CUDA"):
        va.free_pages(a["bt"], a["su"], a["pc"], a["refs"], a["a"])
    with pytest.raises(TypeError):
        va.fork_pages(a["bt"].long(), a["su"], a["pc"], a["refs"], a["a"], a["b"])
    with pytest.raises(ValueError, match="different devices"):
        va.reserve_pages(a["bt"], a["su"], a["pc"], a["refs"], a["new"].to("meta"), a["src"], a["dst"], a["room"])
    with pytest.raises(ValueError, match="CUDA"):
        va.copy_pages(SAME, None, a["a"], a["b"])


@pytest.mark.parametrize("seed", range(20))
def test_oracle_keeps_a_pool(seed):
    """Through random calls: refs are the rows that hold a page, a row's places that it may
    write hold pages of its own, contents follow the copies."""
    r = random.Random(seed)
    B, W, N = 7, 9, 30
    table, used, count, refs = [[0] * W for _ in range(B)], [0] * B, [0] * B, [0] * N
    text = {}                                     # page -> tokens, as a cache holds them
    want = [[] for _ in range(B)]                 # each sequence's tokens
    for _ in range(60):
        what = r.choice(["free", "fork", "reserve", "reserve", "drop"])
        if what == "free":
            s = r.randrange(B)
            pool.free(table, used, count, refs, [s, s])
            want[s] = []
        elif what == "fork":
            p, c = r.sample(range(B), 2)
            if pool.fork(table, used, count, refs, [p], [c]) == 0:
                want[c] = list(want[p])
        elif what == "drop":                      # rejected tokens
            s = r.randrange(B)
            used[s] = max(0, used[s] - r.randrange(20))
            want[s] = want[s][:used[s]]
        else:
            add = [r.choice([0, 1, 5, 20]) if r.random() < 0.6 else 0 for _ in range(B)]
            _, src, dst, room = pool.reserve(table, used, count, refs, add)
            for a, z in zip(src, dst):
                if a >= 0:
                    text[z] = list(text[a])
            for s in range(B):
                if add[s] and room[s] >= used[s] + add[s]:
                    for _ in range(add[s]):
                        page, slot = table[s][used[s] // 16], used[s] % 16
                        assert refs[page] == 1
                        text.setdefault(page, [None] * 16)[slot] = (s, r.random())
                        want[s].append(text[page][slot])
                        used[s] += 1
        held = [page for s in range(B) for page in table[s][:count[s]]]
        assert refs == [held.count(page) for page in range(N)]
        for s in range(B):
            assert [text[table[s][i // 16]][i % 16] for i in range(used[s])] == want[s]
