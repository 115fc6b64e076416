"""Tensors that the append calls write have to give every row (and scale) a place
of its own: two CTAs would write the same bytes otherwise. Host checks only (CPU
tensors, C ABI called directly, before any launch)."""
import pytest
import torch

from test_append_validation import E4, F8, LAYOUT, built, call_kv, call_mla  # noqa: F401

BF = torch.bfloat16


def view(dtype, shape, stride):
    """A tensor with these strides (in elements), on memory that holds it."""
    n = 1 + sum((a - 1) * b for a, b in zip(shape, stride))
    if dtype == F8:
        return torch.zeros(n, dtype=torch.uint8).as_strided(shape, stride).view(F8)
    return torch.zeros(n, dtype=dtype).as_strided(shape, stride)


def cache(stride, dtype=BF, heads=2, width=256):
    return view(dtype, (8, 16, heads, width), (*stride, 1))


OVERLAP = [
    dict(q_out=view(BF, (5, 4, 256), (256, 256, 1))),              # a token's head 1 is the next token's head 0
    dict(q_out=view(BF, (5, 4, 256), (768, 256, 1))),              # the last head is the next token's first
    dict(q_out=view(BF, (5, 4, 256), (256, 1024, 1))),             # tokens inside heads: five of them do not fit
    dict(kc=cache((512, 512, 256))),                               # page stride = slot stride
    dict(vc=cache((512 * 15, 512, 256))),                          # the last slot is the next page's first
    dict(kc=cache((16 * 256, 256, 256))),                          # slot stride = head stride
    dict(E4, ks=view(torch.float32, (8, 2), (1, 1)), vs=torch.ones(8, 2)),
    dict(E4, ks=torch.ones(8, 2), vs=view(torch.float32, (8, 2), (2, 4))),   # pages inside heads, too close
]


@pytest.mark.parametrize("i", range(len(OVERLAP)))
def test_overlapping_rows_are_refused(i):
    assert call_kv(**OVERLAP[i]) == LAYOUT


def test_overlapping_rows_are_refused_latent():
    assert call_mla(q_out=view(BF, (5, 4, 64), (64, 64, 1))) == LAYOUT
    assert call_mla(kc=view(BF, (8, 16, 1, 576), (576, 576, 576, 1))) == LAYOUT
    assert call_mla(kc=view(BF, (8, 16, 1, 576), (15 * 576, 576, 576, 1))) == LAYOUT


def test_views_with_places_of_their_own_pass():
    """Whatever the order of the dimensions, interleaved or padded: past the layout
    checks (the call has no token or no sequence, so nothing is launched)."""
    none = dict(k=torch.zeros(0, 2, 256, dtype=BF), v=torch.zeros(0, 2, 256, dtype=BF), q=None, q_out=None)
    kv = torch.zeros(8, 2, 16, 2, 256, dtype=BF)
    by_head = torch.zeros(8, 16, 2, 2, 256, dtype=BF)
    both = torch.zeros(8, 2, 2)
    for kc, vc in ((kv[:, 0], kv[:, 1]), (by_head[..., 0, :], by_head[..., 1, :]),
                   (cache((256, 8 * 256, 8 * 16 * 256)), cache((16 * 512, 256, 16 * 256))),
                   (cache((1 << 20, 1 << 14, 264)), cache((16 * 512, 512, 256)))):
        assert call_kv(**none, kc=kc, vc=vc) == 0
    for ks, vs in ((both[..., 0], both[..., 1]), (torch.zeros(2, 8).t(), torch.zeros(2, 9).t()[:8]), (torch.zeros(8, 5)[:, 1:3], torch.zeros(8, 2))):
        assert call_kv(**none, **E4, ks=ks, vs=vs) == 0
    empty = dict(bt=torch.zeros(0, 3, dtype=torch.int32), cu=torch.zeros(1, dtype=torch.int32), su=torch.zeros(0, dtype=torch.int32))
    for q in (torch.zeros(4, 5, 256, dtype=BF).transpose(0, 1), torch.zeros(5, 4, 320, dtype=BF)[..., :256], torch.zeros(5, 9, 256, dtype=BF)[:, ::2][:, :4]):
        assert call_kv(**empty, q=q, q_out=q) == 0
    one = dict(k=torch.zeros(0, 1, 256, dtype=BF), v=torch.zeros(0, 1, 256, dtype=BF), q=None, q_out=None)
    assert call_kv(**one, kc=cache((16 * 256, 256, 0), heads=1), vc=cache((16 * 256, 256, 0), heads=1)) == 0
