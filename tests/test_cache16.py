"""The 16-bit paged cache's writer (sdp_cache16_append): refusals on the CPU; on the GPU the rows that it writes against
sdp_qk_norm_rope's (equal, bit for bit) and against the definition in 64 bits, and every other place of the pool as it was.

Tolerance against 64 bits, for a row with norm factor r, channel pair (a, b) and weights w: A x and B x' carry the roundings
of r, of w cos and w' sin, of the cosine and sine themselves and of the products and the sum, each 2^-24 of
r (|w a| + |w' b|) or a few of them (rsqrtf 2^-22, sincospif 2^-22, the mean of squares D / 8 + 5 sums): 2^-18 of it in
all, and half a step of the stored type.
"""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp
from test_cache4 import make_table

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
A = 0x10000


def append_call(**kw):
    from gqa_flash_attention_gb300 import serving
    a = dict(kc=A, vc=2 * A, P=8, page=16, table=3 * A, ts=4, mp=4, q=4 * A, qst=1024, qsh=128, qo=5 * A, qost=1024, qosh=128,
             k=6 * A, kst=256, ksh=128, v=7 * A, vst=256, vsh=128, cu=8 * A, lens=9 * A, nseq=2, tokens=5, pos=10 * A, ps=1,
             p64=0, turns=11 * A, R=64, mscale=1.0, wq=12 * A, wk=13 * A, w32=0, eps=1e-6, il=0, Hq=8, Hkv=2, D=128, dtype=0)
    a.update(kw)
    return serving._lib().sdp_cache16_append(*a.values(), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), sdp.SDP_ERR_UNSUPPORTED),
    (dict(dtype=2), sdp.SDP_ERR_UNSUPPORTED),
    (dict(nseq=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(tokens=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(Hkv=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(Hq=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(P=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(page=24), sdp.SDP_ERR_INVALID_ARG),
    (dict(mp=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(ts=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(R=24), sdp.SDP_ERR_INVALID_ARG),
    (dict(R=144), sdp.SDP_ERR_INVALID_ARG),
    (dict(eps=-1.0), sdp.SDP_ERR_INVALID_ARG),
    (dict(eps=math.nan), sdp.SDP_ERR_INVALID_ARG),
    (dict(mscale=math.inf), sdp.SDP_ERR_INVALID_ARG),
    (dict(kc=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(vc=A), sdp.SDP_ERR_INVALID_ARG),
    (dict(q=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(qo=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(v=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(cu=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(turns=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(kst=260), sdp.SDP_ERR_ALIGNMENT),
    (dict(vsh=132), sdp.SDP_ERR_ALIGNMENT),
    (dict(kc=A + 8), sdp.SDP_ERR_ALIGNMENT),
    (dict(wk=13 * A + 2), sdp.SDP_ERR_ALIGNMENT),
    (dict(pos=10 * A + 4, p64=1), sdp.SDP_ERR_ALIGNMENT),
    (dict(lens=9 * A + 2), sdp.SDP_ERR_ALIGNMENT),
    (dict(mp=1 << 28), sdp.SDP_ERR_OVERFLOW),
    (dict(Hkv=1 << 30), sdp.SDP_ERR_OVERFLOW),
])
def test_append_refuses_before_any_launch(kw, code):
    from gqa_flash_attention_gb300 import build
    build.build()
    assert append_call(**kw) == code


def test_append_of_no_tokens_needs_no_pointers():
    from gqa_flash_attention_gb300 import build
    build.build()
    assert append_call(tokens=0, q=0, k=0, v=0, kc=0, vc=0) == sdp.SDP_OK


def test_cache16_empty_checks():
    for kw in (dict(D=64), dict(page_size=24), dict(num_pages=0), dict(Hkv=0), dict(dtype=torch.float32)):
        with pytest.raises(ValueError):
            sdp.cache16_empty(**{**dict(num_pages=2, Hkv=1, D=128, page_size=16, device="cpu"), **kw})
    c = sdp.cache16_empty(3, 2, 256, 48, torch.float16, device="cpu")
    assert c.k.shape == c.v.shape == (3, 2, 48, 256) and c.k.dtype == torch.float16


# ------------------------------------------------------------------ GPU


def norm_rope64(x, w, pos, freq, R, interleaved, mscale, eps=1e-6):
    """Rows x [T, H, D] in 64 bits, and the size of what their sums add."""
    x = x.double()
    size = x.abs()
    if w is not None:
        r = 1 / torch.sqrt((x ** 2).mean(-1, keepdim=True) + eps)
        x, size = x * r * w.double(), size * r * w.double().abs()
    if R:
        t = pos.double()[:, None] * freq
        c, s = (mscale * torch.cos(t))[:, None], (mscale * torch.sin(t))[:, None]
        i = torch.arange(R // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        y, z = x.clone(), size.clone()
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        z[..., a] = z[..., b] = abs(mscale) * (size[..., a] + size[..., b])
        x, size = y, z
    return x, size


CASES = []
for dt in ("fp16", "bf16"):
    CASES += [
        # lens, new rows, Hq, Hkv, D, page, R, norm, interleaved, positions, dt
        ([1], [1], 1, 1, 128, 16, 128, True, False, None, dt),
        ([17, 16, 0, 33, 500], [1, 1, 0, 1, 1], 8, 2, 128, 16, 128, True, False, None, dt),
        ([40, 7, 200], [40, 3, 130], 7, 1, 256, 48, 64, True, True, None, dt),
        ([300, 20], [300, 0], 6, 3, 128, 64, 96, False, False, "int32", dt),
        ([90, 64, 65], [5, 64, 2], 4, 4, 256, 32, 256, False, True, "int64", dt),
        ([70], [70], 0, 5, 128, 16, 128, True, False, None, dt),          # no queries
        ([33, 100], [32, 100], 16, 2, 256, 256, 0, True, False, None, dt),  # norms alone
        ([129, 5], [1, 5], 3, 3, 128, 16, 0, False, False, None, dt),       # a plain copy
        ([2000, 1500], [2000, 1500], 32, 8, 128, 64, 128, True, False, None, dt),
    ]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new,Hq,Hkv,D,page,R,norm,interleaved,positions,dt", CASES)
def test_append(lens, new, Hq, Hkv, D, page, R, norm, interleaved, positions, dt):
    dtype = DTYPES[dt]
    g = torch.Generator().manual_seed(5 * sum(lens) + D + R)
    table, pool = make_table(lens, page, g)
    behind = 3  # rows behind the last sequence: left as they are
    T = sum(new)
    qkv = torch.randn(T + behind, Hq + 2 * Hkv, D, generator=g).to(dtype)
    cache = sdp.Cache16(*(torch.randn(pool, Hkv, page, D, generator=g).to(dtype).cuda() for _ in range(2)))
    before = sdp.Cache16(*(t.clone() for t in cache))
    w = [(1 + 0.2 * torch.randn(D, generator=g)) for _ in range(2)] if norm else [None, None]
    wt = torch.float32 if page == 48 else dtype
    w = [None if x is None else x.to(wt) for x in w]
    freq = sdp.rope_inv_freq(R, base=5e6)
    rope = sdp.rope_table(freq, mscale=1.1, device="cuda") if R else None
    place = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)] + [torch.zeros(behind, dtype=torch.long)])
    given = None
    at = place
    if positions:
        at = torch.randint(0, 1000000, (T + behind,), generator=g)
        given = at.to(getattr(torch, positions)).cuda()
    cu = torch.tensor([0, *torch.tensor(new).cumsum(0).tolist()], dtype=torch.int32).cuda()
    x = qkv.cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    wc = [None if t is None else t.cuda() for t in w]
    q_out = torch.full((T + behind, Hq, D), 7.0, dtype=dtype, device="cuda") if Hq else None
    got = sdp.cache16_append(cache, k, v, cu, torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), rope=rope,
                             q=q if Hq else None, positions=given, q_weight=wc[0] if Hq else None, k_weight=wc[1],
                             interleaved=interleaved, q_out=q_out)
    assert sdp.poll_status() == sdp.SDP_OK
    assert got is q_out
    # the same rows by sdp_qk_norm_rope, and nothing else touched
    if Hq:
        fq, fk = sdp.qk_norm_rope(q, k, at.cuda(), rope, q_weight=wc[0], k_weight=wc[1], interleaved=interleaved)
        assert torch.equal(got[:T], fq[:T]) and (got[T:] == 7).all()
    else:
        fk, _ = sdp.qk_norm_rope(k, None, at.cuda(), rope, q_weight=wc[1], interleaved=interleaved)
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(new))
    ids, off = table[seq, place[:T] // page].long().cuda(), (place[:T] % page).cuda()
    for pool_t, was, rows in ((cache.k, before.k, fk), (cache.v, before.v, v)):
        was[ids, :, off] = rows[:T]
        assert torch.equal(pool_t, was)
    for rows, wx, res in ((qkv[:T, :Hq], w[0], got), (qkv[:T, Hq:Hq + Hkv], w[1], cache.k[ids, :, off])):
        if res is None:
            continue
        ref, size = norm_rope64(rows, wx, at[:T], freq, R, interleaved, 1.1)
        off64 = (res[:T].double().cpu() - ref).abs()
        assert (off64 <= torch.finfo(dtype).eps / 2 * ref.abs() + 2.0 ** -18 * size + 2.0 ** -25).all(), off64.max()


def small(dtype=torch.float16, pages=8, Hkv=2, D=128, page=16):
    c = sdp.cache16_empty(pages, Hkv, D, page, dtype)
    x = torch.randn(8, 3 * Hkv, D, device="cuda").to(dtype)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(2, -1)
    return c, x[:, :Hkv], x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:], table


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
def test_append_reports_bad_input():
    c, q, k, v, table = small()
    ok = (i32(0, 4, 8), i32(9, 40), table)
    bad_pages = table.clone()
    bad_pages[1, 2] = 8  # holds tokens 32 .. 47 of the second sequence
    for cu, lens, tab, code in (
            (i32(0, 4, 9), ok[1], table, sdp.SDP_ERR_BAD_SEQLENS),    # past the tokens
            (i32(-1, 4, 8), ok[1], table, sdp.SDP_ERR_BAD_SEQLENS),
            (i32(0, 6, 4), ok[1], table, sdp.SDP_ERR_BAD_SEQLENS),    # decreasing
            (ok[0], i32(3, 40), table, sdp.SDP_ERR_BAD_SEQLENS),      # shorter than its new rows
            (ok[0], i32(9, 65), table, sdp.SDP_ERR_BAD_SEQLENS),      # longer than its pages
            (ok[0], i32(9, -2 ** 31), table, sdp.SDP_ERR_BAD_SEQLENS),
            (ok[0], ok[1], bad_pages, sdp.SDP_ERR_BAD_PAGES)):
        for t in c:
            t.zero_()
        out = torch.full_like(q, 5).contiguous()
        sdp.cache16_append(c, k, v, cu, lens, tab, q=q, q_out=out)
        assert sdp.poll_status() == code
        if code == sdp.SDP_ERR_BAD_PAGES:  # the queries need no page; the other sequence is written
            assert torch.equal(out, q) and torch.equal(c.v[0, :, 5:9].transpose(0, 1), v[:4])
            assert int((c.v != 0).any(-1).sum()) == 4 * 2
    assert sdp.poll_status() == sdp.SDP_OK
    sdp.cache16_append(c, k, v, *ok)
    assert sdp.poll_status() == sdp.SDP_OK


@pytest.mark.gpu
def test_append_refusals_of_the_binding():
    c, q, k, v, table = small()
    cu, lens = i32(0, 4, 8), i32(9, 40)
    rope = sdp.rope_table(sdp.rope_inv_freq(64), device="cuda")
    good = dict(cache=c, k=k, v=v, cu_seqlens=cu, cache_lens=lens, block_table=table)
    for kw in (dict(cache=(c.k,)), dict(cache=sdp.Cache16(c.k, c.v.bfloat16())), dict(k=k.bfloat16()), dict(v=v[:4]),
               dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu[:2]), dict(cache_lens=lens[:1]), dict(block_table=table.long()),
               dict(q=q[:4]), dict(q=q.float()), dict(q_out=q), dict(q=q, q_out=q[:4]), dict(q_weight=torch.ones(128).cuda()),
               dict(k_weight=torch.ones(64).cuda()), dict(positions=cu), dict(rope=rope, positions=cu),
               dict(rope=rope, positions=torch.zeros(8).cuda()), dict(rope=(1,)), dict(interleaved=torch.ones(2)),
               dict(k=k.cpu()), dict(stream="x"), dict(k=k.clone().requires_grad_())):
        with pytest.raises(ValueError):
            sdp.cache16_append(**{**good, **kw})
    with pytest.raises(sdp.SdpError):  # channels that do not lie on 16 bytes
        sdp.cache16_append(**{**good, "k": torch.zeros(8, 2, 132, device="cuda").half()[..., :128]})
    torch.cuda.synchronize()
    assert (c.k == 0).all() and sdp.poll_status() == sdp.SDP_OK


@pytest.mark.gpu
def test_append_in_place_and_no_sequences():
    c, q, k, v, table = small()
    cu, lens = i32(0, 4, 8), i32(9, 40)
    rope = sdp.rope_table(sdp.rope_inv_freq(128), device="cuda")
    want = sdp.cache16_append(c, k, v, cu, lens, table, rope=rope, q=q)
    assert sdp.cache16_append(c, k, v, cu, lens, table, rope=rope, q=q, q_out=q) is q
    assert torch.equal(q, want)
    before = c.k.clone()
    sdp.cache16_append(c, k, v, i32(0), i32(), table[:0])
    empty = sdp.cache16_append(c, k[:0], v[:0], i32(0, 0, 0), lens, table, q=q[:0])
    assert empty.shape == (0, 2, 128) and torch.equal(c.k, before) and sdp.poll_status() == sdp.SDP_OK


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [False, True])
def test_positions_without_a_rotation_change_nothing(norm):
    """As a model passes them to every layer, of which some rotate nothing."""
    c, q, k, v, table = small()
    cu, lens = i32(0, 4, 8), i32(9, 40)
    w = torch.linspace(0.5, 1.5, 128, device="cuda").half() if norm else None
    want = sdp.cache16_append(c, k, v, cu, lens, table, q=q, q_weight=w, k_weight=w)
    before = c.k.clone()
    for dtype in (torch.int32, torch.int64):
        c.k.zero_()
        got = sdp.cache16_append(c, k, v, cu, lens, table, q=q, q_weight=w, k_weight=w,
                                 positions=torch.arange(1000, 1008, device="cuda", dtype=dtype))
        assert torch.equal(got, want) and torch.equal(c.k, before)
    assert sdp.poll_status() == sdp.SDP_OK
