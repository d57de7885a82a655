"""Corners of the 16-bit paged cache: the start of a call whose entries fill every thread, limits of the arguments, offsets that
no row belongs to, groups that shrink to one sequence, values that are not finite, many heads behind a prefix."""

import pytest
import torch

import gqa_flash_attention_gb300 as sdp
from test_cache16_attn import Batch, c_call


@pytest.mark.parametrize("kw", [
    # a box is looked up from up to 32 tiles behind the last key on: the largest tables that leave those no room
    dict(page=128, mp=(2 ** 31 - 384) // 128), dict(page=128, pp=(2 ** 31 - 384) // 128),
    dict(page=128, mp=(2 ** 31 - 4096) // 128), dict(page=128, pp=(2 ** 31 - 4096) // 128),
    dict(page=16, mp=(2 ** 31 - 4096) // 16), dict(page=2 ** 30 - 512, mp=2, ng=0)])
def test_tables_of_almost_two_to_the_31_keys_are_refused(kw):
    from gqa_flash_attention_gb300 import build
    build.build()
    assert c_call(**{**dict(nseq=1, Hq=1, Hkv=1), **kw}) == sdp.SDP_ERR_OVERFLOW


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
def test_starts_of_many_entries(D):
    """Each call's offsets pass through shared memory where its first copies land next: 512 entries, one a thread, all of them
    short, so that a CTA copies as soon as its first unit is known. The same bits from 200 calls back to back."""
    b = Batch([1 + i % 40 for i in range(512)], [0], [], 1, 2, 2, D, 16, torch.bfloat16)
    a = b.args()
    ws = torch.empty(sdp.cache16_workspace_bytes(512, 1, 2, 2, D, torch.bfloat16), dtype=torch.uint8, device="cuda")
    want = sdp.fwd_cache16(**a, workspace=ws)
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(*want)
    outs = [(torch.full_like(want[0], 9), torch.full_like(want[1], 9)) for _ in range(200)]
    for o, lse in outs:
        sdp.fwd_cache16(**a, out=o, lse=lse, workspace=ws)
    assert sdp.poll_status() == sdp.SDP_OK
    for o, lse in outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
def test_waits_for_the_first_unit_that_run_out(D):
    """No unit is published: every warp gives up before it has one, looks nothing up, and the next call is right."""
    b = Batch([500, 300, 420, 290], [0, 3], [280], 1, 8, 2, D, 32, torch.bfloat16)
    a = b.args()
    want = sdp.fwd_cache16(**a)
    assert sdp.poll_status() == sdp.SDP_OK
    old = sdp.set_wait_timeout_ms(20)
    sdp.set_debug_flags(256)
    try:
        sdp.fwd_cache16(**a)
        assert sdp.poll_status() == sdp.SDP_ERR_DEVICE_TIMEOUT
    finally:
        sdp.set_debug_flags(0)
        sdp.set_wait_timeout_ms(old)
    o, lse = sdp.fwd_cache16(**a)
    assert sdp.poll_status() == sdp.SDP_OK and torch.equal(o, want[0]) and torch.equal(lse, want[1])
