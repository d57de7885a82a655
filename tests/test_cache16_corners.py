"""Corners of the 16-bit paged cache: the start of a call whose entries fill every thread, limits of the arguments, offsets that
no row belongs to, groups that shrink to one sequence, values that are not finite, many heads behind a prefix."""

import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp
from test_cache16_attn import DTYPES, Batch, c_call


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kw", [
    # a box is looked up from up to 32 tiles behind the last key on: the largest tables that leave those no room
    dict(page=128, mp=(2 ** 31 - 384) // 128), dict(page=128, pp=(2 ** 31 - 384) // 128),
    dict(page=128, mp=(2 ** 31 - 4096) // 128), dict(page=128, pp=(2 ** 31 - 4096) // 128),
    dict(page=16, mp=(2 ** 31 - 4096) // 16), dict(page=2 ** 30 - 512, mp=2, ng=0)])
def test_tables_of_almost_two_to_the_31_keys_are_refused(kw):
    from gqa_flash_attention_gb300 import build
    build.build()
    assert c_call(**{**dict(nseq=1, Hq=1, Hkv=1), **kw}) == sdp.SDP_ERR_OVERFLOW


@pytest.mark.parametrize("scale", [3e38, -3e38, 2.36e38, math.inf])
def test_scales_that_leave_fp32_in_powers_of_two_are_refused(scale):
    """They would be multiplied as infinities: a score of 0 as NaN."""
    from gqa_flash_attention_gb300 import build
    build.build()
    assert c_call(scale=scale) == sdp.SDP_ERR_INVALID_ARG


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


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [64, 75, 600])
@pytest.mark.parametrize("rows,D", [(1, 128), (3, 256)])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_groups_of_one_sequence(prefix, rows, D, dt):
    """Their prefixes are read from the prefix's pages, as those of larger groups: their own tables have none for the pages
    that it fills, and where it ends inside a page their own page holds NaN and infinities up to there."""
    b = Batch([prefix + 70, prefix + rows - 1, prefix + 1000], [0, 3], [prefix], rows, 8, 2, D, 16, DTYPES[dt])
    assert (b.table[:, :prefix // 16] == -7).all()
    a = b.args()
    a["prefix_table"], a["prefix_lens"] = a["prefix_table"].repeat(3, 1), i32(prefix, prefix, prefix)
    a["cu_groups"] = i32(0, 1, 2, 3)
    o, lse = sdp.fwd_cache16(**a)
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(o, lse)


@pytest.mark.gpu
def test_a_captured_step_whose_group_shrinks_to_one():
    b = Batch([300, 333, 290], [0, 3], [139], 2, 8, 2, 128, 48, torch.bfloat16)
    a = b.args()
    out, lse = torch.zeros_like(a["q"]), torch.zeros(a["q"].shape[:-1], device="cuda")
    ws = torch.empty(sdp.cache16_workspace_bytes(3, 2, 8, 2, 128, torch.bfloat16, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdp.fwd_cache16(**a, out=out, lse=lse, workspace=ws)
    for left in (3, 2, 1, 0):  # sequences: the others end, and their places are padding
        a["cu_groups"][1] = left
        a["cache_lens"][left:] = 0
        out.fill_(5)
        graph.replay()
        assert sdp.poll_status() == sdp.SDP_OK
        b.check(out, lse, only=range(left))
        assert (out[left:] == 0).all() and (lse[left:] == -math.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D,G,P", [(128, 4, 300), (256, 16, 300), (128, 1, 12000)])
def test_an_infinite_draft_behind_a_prefix_of_far_larger_scores(D, G, P):
    """The prefix's keys score 2^250 times the others in weight, which leaves those no fp32 weight at all: an infinity or a NaN in
    a drafted token's V, whose weight is positive, decides its channel of the rows that see it all the same."""
    rows, page, loud = 3, 16, 11.0 * math.sqrt(D)
    b = Batch([P + 9, P + 40], [0, 2], [P], rows, G, 1, D, page, torch.bfloat16)
    b.q[..., 7] = 16.0
    t = torch.arange(P)
    b.k[b.prefix_table[0, t // page].long(), :, t % page, 7] = loud
    for s, n in enumerate(b.lens):
        t = torch.arange(P, n)
        b.k[b.table[s, t // page].long(), :, t % page, 7] = 0
        b.rows_kv[s][0][:P, :, 7], b.rows_kv[s][0][P:, :, 7] = loud, 0
    want, lse = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(want, lse)
    for s, back, c, x in ((0, 2, 5, math.inf), (0, 1, 9, math.nan), (1, 1, 64, -math.inf), (1, 3, D - 1, math.inf)):
        t = b.lens[s] - back
        b.v[int(b.table[s, t // page]), 0, t % page, c] = x
        want[s, rows - back:, :, c] = x
    o, l2 = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK and torch.equal(l2, lse)
    same = (o == want) | (o.isnan() & want.isnan())
    assert same.all(), same.logical_not().nonzero()[:4]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,Hkv,D", [(1, 1, 128), (1, 1, 256), (1, 2, 256), (2, 1, 128), (3, 4, 128)])
def test_appending_few_rows_checks_all_offsets(tokens, Hkv, D):
    """A call of fewer than four warps' work: bad offsets of sequences that none of its rows belongs to are reported, wherever
    they stand among the sequences'."""
    nseq = 300
    c = sdp.cache16_empty(8, Hkv, D, 16, torch.float16)
    k = torch.ones(tokens, Hkv, D, dtype=torch.float16, device="cuda")
    table = torch.zeros(nseq, 1, dtype=torch.int32, device="cuda")
    lens = torch.full((nseq,), 16, dtype=torch.int32, device="cuda")
    good = torch.full((nseq + 1,), tokens, dtype=torch.int32, device="cuda")
    good[0] = 0
    sdp.cache16_append(c, k, k, good, lens, table)
    assert sdp.poll_status() == sdp.SDP_OK
    for at in range(1, nseq + 1):
        cu = good.clone()
        cu[at] = tokens + 1
        sdp.cache16_append(c, k, k, cu, lens, table)
        assert sdp.poll_status() == sdp.SDP_ERR_BAD_SEQLENS, at


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["k", "v"])
def test_caches_that_require_grad_are_refused(which):
    """As learned prefixes would: no gradient would come back. Without grad mode they are as good as others."""
    b = Batch([40, 50], [0], [], 1, 2, 1, 128, 16, torch.float16)
    a = b.args()
    want = sdp.fwd_cache16(**a)
    getattr(a["cache"], which).requires_grad_()
    new = dict(cu_seqlens=i32(0, 1, 1), cache_lens=a["cache_lens"], block_table=a["block_table"])
    row = torch.ones(1, 1, 128, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        sdp.fwd_cache16(**a)
    with pytest.raises(ValueError):
        sdp.cache16_append(a["cache"], row, row, **new)
    with torch.no_grad():
        got = sdp.fwd_cache16(**a)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        sdp.cache16_append(a["cache"], row, row, **new)
    assert sdp.poll_status() == sdp.SDP_OK


@pytest.mark.gpu
@pytest.mark.parametrize("lens,cu,prefix,rows,Hq,Hkv,D,page,dt", [
    ([300, 333, 290], [0, 3], [139], 3, 200, 1, 128, 48, "bf16"),  # a prefix that ends inside a page
    ([300, 333, 141, 2, 500], [0, 3, 4, 5], [139, 50, 480], 2, 400, 2, 256, 32, "fp16"),
    ([900, 700], [0, 2], [640], 1, 129, 1, 256, 64, "bf16"),
])
def test_more_heads_than_a_block_behind_a_prefix(lens, cu, prefix, rows, Hq, Hkv, D, page, dt):
    """More than 128 query heads a KV head: blocks of heads, the last one not full, in both kinds of problems and in the join."""
    b = Batch(lens, cu, prefix, rows, Hq, Hkv, D, page, DTYPES[dt])
    o, lse = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("D,G", [(128, 4), (256, 16)])
def test_values_of_a_prefix_that_are_not_finite(D, G, dt):
    """An infinity or a NaN in the V of a key that all rows see (with a weight that the 16-bit type holds) reaches its channel
    of the rows of its group, and nothing else."""
    page, P = 16, 200
    b = Batch([230, 205, 900, 300], [0, 3], [P], 2, G, 1, D, page, DTYPES[dt])
    want, lse = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK
    for t, c, x in ((0, 3, math.inf), (130, D - 1, -math.inf), (P - 1, 64, math.nan)):
        b.v[int(b.prefix_table[0, t // page]), 0, t % page, c] = x
        want[:3, :, :, c] = x
    t = 250  # one of the sequence in no group
    b.v[int(b.table[3, t // page]), 0, t % page, 7] = math.inf
    want[3, :, :, 7] = math.inf
    o, l2 = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK and torch.equal(l2, lse)
    same = (o == want) | (o.isnan() & want.isnan())
    assert same.all(), same.logical_not().nonzero()[:4]
