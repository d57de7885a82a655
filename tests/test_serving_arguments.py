"""Arguments of the serving operators that are of no use as what they stand for: a ValueError, before any launch."""
import pytest
import torch

import gqa_flash_attention_gb300 as sdp


@pytest.mark.gpu
def test_truth_values():
    both = torch.ones(2)  # neither true nor false
    x = torch.randn(1, 2, 64, 128, device="cuda").half()
    out = torch.full_like(x, 3)
    t = x[0].transpose(0, 1).contiguous()
    cu = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    cache, table = sdp.cache4_empty(4, 2, 128, 16), torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    lens = torch.tensor([64], dtype=torch.int32, device="cuda")
    for call in (lambda: sdp.fwd_window(x, x, x, 9, out=out, return_lse=both),
                 lambda: sdp.fwd_varlen_window(t, t, t, cu, cu, 64, 9, out=out[0].transpose(0, 1).contiguous(), return_lse=both),
                 lambda: sdp.fwd_cache4(t[:1], cache, lens, table, out=out[0, :, 0][None].contiguous(), return_lse=both),
                 lambda: sdp.qk_norm_rope(x, None, None, None, interleaved=both, q_out=out)):
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()
    assert (out == 3).all() and sdp.poll_status() == sdp.SDP_OK
    o, lse = sdp.fwd_window(x, x, x, 9, return_lse=0)  # what Python takes for true or false is
    assert lse is None


def test_types_of_a_workspace():
    for dtype in (torch.float32, None):
        with pytest.raises(ValueError):
            sdp.cache4_workspace_bytes(1, 1, 8, 2, 128, dtype)
