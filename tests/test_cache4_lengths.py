"""cache4_append with lengths at the ends of 32 bits, over a block table as wide as the call takes."""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-2 ** 31, -2 ** 31 + 50, -1, 0, 99])
def test_a_length_below_its_new_rows_is_bad_whatever_its_sign(bad):
    wide = (2 ** 31 - 1) // 16
    table = torch.zeros(1, wide, dtype=torch.int32, device="cuda")
    cache = sdp.cache4_empty(7, 1, 128, 16)
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(math.nan)
    before = [t.clone() for t in cache]
    x = torch.randn(100, 1, 128, device="cuda").half()
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    sdp.cache4_append(cache, x, x, cu, torch.tensor([bad], dtype=torch.int32, device="cuda"), table)
    assert sdp.poll_status() == sdp.SDP_ERR_BAD_SEQLENS
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, before))
    # the last tokens that a table can hold
    n = wide * 16
    table[0, -7:] = torch.arange(7, dtype=torch.int32, device="cuda")
    sdp.cache4_append(cache, x, x, cu, torch.tensor([n], dtype=torch.int32, device="cuda"), table)
    assert sdp.poll_status() == sdp.SDP_OK
    scales = cache.k_scales.view(7 * 16, -1)
    assert torch.isfinite(scales[12:].float()).all() and torch.isnan(scales[:12].float()).all()
