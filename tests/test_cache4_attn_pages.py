"""fwd_cache4 where a manager has given up the pages that no row sees any more: their entries of the block table
are not read. Tolerances as in test_cache4_attn.
"""
import pytest
import torch

import gqa_flash_attention_gb300 as sdp
from test_cache4_attn import DTYPES, check, fill

CASES = []
for dt, D in (("fp16", 128), ("bf16", 256)):
    for page in (16, 32, 48, 64, 80):
        CASES += [
            # lens, rows, Hq, Hkv, window, sinks
            ([900, 33, 257, 0, 16, 640], 1, 8, 2, 50, 4, page, D, dt),
            ([900, 33, 257, 5, 16, 641], 5, 8, 1, 33, 0, page, D, dt),     # several chunks of columns
            ([1000, 500, 129, 700, 48, 96], 1, 4, 4, 1, 17, page, D, dt),
            ([1000, 500, 129, 700, 48, 96], 3, 4, 4, 16, 49, page, D, dt),
            ([900, 333, 400], 2, 8, 2, 50, 40, page, D, dt),               # a tile across pages 0 and 1 of 48
            ([900, 333, 400], 1, 8, 2, 50, 70, page, D, dt),               # and of 80
            ([770, 385, 257, 400], 1, 4, 2, 100, 0, page, D, dt),          # first windows' tiles across pages
            ([770, 385, 257, 400], 4, 4, 2, 28, 1, page, D, dt),
        ]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,rows,Hq,Hkv,window,sinks,page,D,dt", CASES)
def test_pages_that_no_row_sees_are_not_looked_up(lens, rows, Hq, Hkv, window, sinks, page, D, dt):
    g = torch.Generator().manual_seed(page + rows)
    dtype = DTYPES[dt]
    cache, table, ks, vs = fill(lens, Hkv, D, page, dtype, g)
    gone = 0
    for s, n in enumerate(lens):
        t = torch.arange(n)
        seen = (t >= n - rows - window + 1) | (t < sinks)
        for x in range(-(-n // page)):
            if not seen[x * page:(x + 1) * page].any():
                table[s, x] = (-1, 10 ** 6)[x % 2]
                gone += 1
    assert gone > 5
    q = torch.randn(len(lens), rows, Hq, D, generator=g).to(dtype).cuda()
    o, lse = sdp.fwd_cache4(q, cache, torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), window=window, sinks=sinks)
    assert sdp.poll_status() == sdp.SDP_OK
    check(q, o, lse, lens, ks, vs, dtype, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 48, 64])
def test_a_seen_page_outside_the_pool_is_still_reported(page):
    g = torch.Generator().manual_seed(page)
    cache, table, _, _ = fill([900], 1, 128, page, torch.float16, g)
    q = torch.randn(1, 1, 4, 128, generator=g).half().cuda()
    dl = torch.tensor([900], dtype=torch.int32).cuda()
    for x in (0, 899 // page, (900 - 50) // page):  # the sinks', the last, the first of the window
        t = table.clone()
        t[0, x] = -1
        sdp.fwd_cache4(q, cache, dl, t.cuda(), window=50, sinks=4)
        assert sdp.poll_status() == sdp.SDP_ERR_BAD_PAGES
