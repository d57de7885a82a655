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
