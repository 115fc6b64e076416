"""append_kv with norms of queries and keys, against the fp64 oracle: every cache
kind, both weight types, with and without a rotation, one of the two norms alone."""
import numpy as np
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from append_util import Batch, check_rotated, check_store, decode, expect, gpu, pair_size, raw
from oracle.append_fp64 import rotated

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "scaled"]

# The norm's fp32 steps ahead of the rotation: a sum of 256 squares (13 roundings deep, half of
# it through the root), the mean and eps (1), the root (2 ulp: 4), w + offset, x r, x r w:
# at most 16 * 2^-24 of a normalised value; the rotation's four beside that are what
# append_util allows. Together 5 times its FP32 of the rows' largest |x1| + |x2|.
STEPS = 5


def weights(seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(256, generator=g)).to(dtype)


def normed(x, w, eps, offset):
    y = decode(x)
    with np.errstate(invalid="ignore"):
        return y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps) * (w.double().numpy() + offset)


def turned(b, y):
    y = y.copy()
    for s in range(len(b.used)):
        a, z = int(b.cu[s]), int(b.cu[s + 1])
        for t in range(z - a):
            y[a + t] = rotated(y[a + t], None if b.cos_sin is None else b.cos_sin.numpy(), b.rope_position(s, t, a + t), b.interleaved)
    return y


def check(b, qw, kw, eps=1e-6, offset=0.0, in_place=False, stream=None):
    caches, scales = [gpu(c) for c in b.caches], [gpu(s) for s in b.scales]
    q = gpu(b.q) if b.cos_sin is not None or qw is not None else None
    q_out = None if q is None else q if in_place else torch.full_like(q, 7.0)
    before = None if q is None else q_out.cpu()
    va.append_kv(gpu(b.k), gpu(b.v), caches[0], caches[1], gpu(b.block_table), gpu(b.cu), gpu(b.used), q=q, q_out=q_out,
                 cos_sin=gpu(b.cos_sin), interleaved=b.interleaved, k_descale=gpu(b.descales[0]), v_descale=gpu(b.descales[1]),
                 k_scales=scales[0], v_scales=scales[1], q_norm=gpu(qw), k_norm=gpu(kw), norm_eps=eps, norm_offset=offset,
                 stream=stream)
    torch.cuda.synchronize()
    if q is not None:
        want = turned(b, normed(b.q, qw, eps, offset) if qw is not None else decode(b.q))
        placed = b.placed()
        assert (raw(q_out)[~placed] == raw(before)[~placed]).all(), "a row without a position changed"
        got, w = decode(q_out)[placed], want[placed]
        tol = 2.0 ** -8 * np.abs(w) + STEPS * 4 * 2.0 ** -24 * pair_size(w)[..., None]
        assert (np.abs(got - w) <= tol).all(), f"worst {np.abs(got - w).max()}"
    k = normed(b.k, kw, eps, offset) if kw is not None else decode(b.k)
    size = STEPS * pair_size(k).max(initial=0.0)
    check_store(b.caches[0], caches[0], expect(b, turned(b, k), 0), scales[0], b.descales[0], size)
    check_store(b.caches[1], caches[1], expect(b, decode(b.v), 1), scales[1], b.descales[1], pair_size(decode(b.v)).max(initial=0.0))
    return q_out, caches, scales


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("q,kv,hq,hkv,rot", [([4, 2], [1024, 769], 16, 1, 256), ([3, 0, 4, 1, 2], [20, 5, 18, 0, 2], 12, 3, 128),
                                            ([37, 16, 1, 130, 15], [37, 48, 300, 141, 31], 5, 1, 64), ([1], [1], 2, 2, 8)])
def test_norm(kind, interleaved, dtype, q, kv, hq, hkv, rot):
    b = Batch(q, kv, hq, hkv, kind, rot, 17 + rot, tail=1, interleaved=interleaved)
    check(b, weights(1, dtype), weights(2, dtype), eps=1e-5)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("which", ["q", "k", "mixed", "no rotation", "offset", "in place"])
def test_forms(kind, which):
    b = Batch([5, 20], [9, 41], 3, 1, kind, 0 if which == "no rotation" else 64, 23)
    qw = None if which == "k" else weights(3, torch.bfloat16)
    kw = None if which == "q" else weights(4, torch.float32 if which == "mixed" else torch.bfloat16)
    check(b, qw, kw, offset=1.0 if which == "offset" else 0.0, in_place=which == "in place")


def test_rows_of_zeros_and_of_extremes():
    """0 / sqrt(eps) is 0; tiny and huge rows come out at the weights' size."""
    b = Batch([6], [6], 2, 1, "bf16", 64, 3)
    b.q[0] = 0
    b.k[1] = 0
    b.q[2] = 2.0 ** -60
    b.k[3] *= 2.0 ** 50
    b.k[4] *= 2.0 ** -50
    check(b, weights(5, torch.bfloat16), weights(6, torch.bfloat16), eps=2.0 ** -130)


def test_other_stream_and_graph():
    b = Batch([3, 2], [50, 17], 8, 2, "scaled", 128, 9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    check(b, weights(7, torch.bfloat16), weights(8, torch.bfloat16), stream=s)
    t = {k: gpu(getattr(b, k)) for k in ("q", "k", "v", "block_table", "cu", "used", "cos_sin")}
    caches, scales = [gpu(c) for c in b.caches], [gpu(x) for x in b.scales]
    out, w = torch.zeros_like(t["q"]), gpu(weights(7, torch.bfloat16))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        va.append_kv(t["k"], t["v"], *caches, t["block_table"], t["cu"], t["used"], q=t["q"], q_out=out, cos_sin=t["cos_sin"],
                     k_scales=scales[0], v_scales=scales[1], q_norm=w, k_norm=w)
    g.replay()
    torch.cuda.synchronize()
    eager = [gpu(c) for c in b.caches], [gpu(x) for x in b.scales], torch.zeros_like(out)
    va.append_kv(t["k"], t["v"], *eager[0], t["block_table"], t["cu"], t["used"], q=t["q"], q_out=eager[2], cos_sin=t["cos_sin"],
                 k_scales=eager[1][0], v_scales=eager[1][1], q_norm=w, k_norm=w)
    torch.cuda.synchronize()
    assert torch.equal(out, eager[2]) and all((raw(x) == raw(y)).all() for x, y in zip(caches, eager[0]))
    assert all(torch.equal(x, y) for x, y in zip(scales, eager[1]))
