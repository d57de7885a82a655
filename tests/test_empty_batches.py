"""The serving operators on batches that hold nothing of a kind: no key at all, no sequence at all."""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[5], [300, 0, 129], [40] * 400])
@pytest.mark.parametrize("D,dtype,Hq", [(128, torch.float16, 4), (256, torch.bfloat16, 4), (256, torch.float16, 3)])
@pytest.mark.parametrize("flags", [0, 32], ids=["compact", "full_grid"])
def test_a_packed_window_batch_without_a_key(lens, D, dtype, Hq, flags):
    T = sum(lens)
    q = torch.randn(T, Hq, D, device="cuda").to(dtype)
    kv = torch.empty(0, 1, D, device="cuda", dtype=dtype)
    cq = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    ck = torch.zeros_like(cq)
    buf = torch.full((T + 1, Hq, D), 7.0, device="cuda", dtype=dtype)
    old = sdp.set_debug_flags(flags)
    try:
        o, lse = sdp.fwd_varlen_window(q, kv, kv, cq, ck, max(lens), 64, sinks=2, out=buf[:T])
        assert sdp.poll_status() == sdp.SDP_OK
        assert (o == 0).all() and (lse == -math.inf).all() and (buf[T] == 7).all()
        o, none = sdp.fwd_varlen_window(q, kv, kv, cq, ck, max(lens), 64, return_lse=False)
        assert sdp.poll_status() == sdp.SDP_OK and none is None and (o == 0).all()
        ck[-1] = 1  # a key that is not there
        sdp.fwd_varlen_window(q, kv, kv, cq, ck, max(lens), 64)
        assert sdp.poll_status() == sdp.SDP_ERR_BAD_SEQLENS
    finally:
        sdp.set_debug_flags(old)


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [0, 3])
def test_a_cache_batch_without_a_sequence(pages):
    """Rows in no sequence are left out, as they are behind the last one; attention does the same."""
    cache = sdp.cache4_empty(4, 2, 128, 16)
    before = [t.clone() for t in cache]
    table = torch.empty(0, pages, dtype=torch.int32, device="cuda")
    cu, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    for n in (0, 5):
        x = torch.randn(n, 2, 128, device="cuda").half()
        sdp.cache4_append(cache, x, x, cu, lens, table)
        out = torch.full_like(x, 3)
        k, v = sdp.cache4_gather(cache, cu, table, n, dtype=torch.float16, k_out=out)
        assert k is out and v.shape == x.shape and (k == 3).all()
    o, lse = sdp.fwd_cache4(torch.empty(0, 8, 128, device="cuda", dtype=torch.float16), cache, lens, table)
    assert o.shape == (0, 8, 128) and lse.shape == (0, 8)
    assert sdp.poll_status() == sdp.SDP_OK
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    with pytest.raises(ValueError):  # offsets of one sequence
        sdp.cache4_append(cache, x, x, torch.zeros(2, dtype=torch.int32, device="cuda"), lens, table)
