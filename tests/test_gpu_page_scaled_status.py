"""Page-scaled calls whose bounded waits run out say so: to the caller's workspace,
or without one (the call's own is gone by then) to the library's status word."""
import pytest
import torch

import speculative_decoding_verify_split_gb300 as va
from speculative_decoding_verify_split_gb300.workloads import make_mla_workload, make_workload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mla", [False, True])
def test_waits_that_run_out(mla):
    """With a limit of 1 ns; without a workspace the library's word has the bits,
    with one that one alone."""
    q, kv = [4, 2, 3], [2500, 700, 130]
    w = (make_mla_workload(q, kv, 16, "fp8_e4m3", seed=31) if mla else make_workload(q, kv, 16, 1, "fp8_e4m3", seed=32)).to("cuda")
    one = torch.ones((w.kv_cache if mla else w.k_cache).shape[0], 1, device="cuda")

    def call(splits, ws=None):
        tail = (w.block_table, w.cu_seqlens_q, w.seqused_k, w.max_seqlen_q, w.max_seqlen_k, w.softmax_scale)
        if mla:
            return va.verify_attn_mla_scaled(w.q, w.kv_cache, one, *tail, workspace=ws, num_splits=splits)
        return va.verify_attn_scaled(w.q, w.k_cache, w.v_cache, one, one, *tail, workspace=ws, num_splits=splits)

    size = va.mla_workspace_size(w.q, w.seqused_k, w.max_seqlen_q, w.max_seqlen_k) if mla else \
        va.workspace_size(w.q, w.k_cache, w.seqused_k, w.max_seqlen_q, w.max_seqlen_k)
    ws = torch.zeros(size + 256, dtype=torch.uint8, device="cuda")
    va.last_device_error()
    splits = (0, 1, 5)                           # clusters, one CTA, a few
    ref = [call(s) for s in splits]
    assert va.last_device_error() == 0
    for given in (None, ws):
        va.set_wait_limit(1)
        try:
            for s in splits:
                call(s, given)
            torch.cuda.synchronize()
        finally:
            va.set_wait_limit(0)
        if given is not None:
            assert va.last_device_error() == 0
        assert va.last_device_error(given) != 0 and va.last_device_error(given) == 0
        assert all(torch.equal(call(s, given), r) for s, r in zip(splits, ref)) and va.last_device_error(given) == 0
