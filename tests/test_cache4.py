"""The 4-bit paged cache: sdp_cache4_append and sdp_cache4_gather.

Refusals on the CPU. On the GPU the written codes and scales are compared with the definition
evaluated in exact rational steps of fp32 (the quotient correctly rounded), so they have to be
equal; and the gathered rows with scale * code + bias in 64 bits: half a step of the stored type
plus the fp32 sum's rounding (2^-24 of the result; the product of 8 and 4 bits is exact).
"""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def quantise(x):
    """Codes [..., D/2] and (scale, bias) [..., D/64, 2] of rows x [..., D] (CPU: divisions are IEEE)."""
    x = x.float().unflatten(-1, (-1, 64))
    bias = x.amin(-1).bfloat16()
    scale = ((x.amax(-1) - bias.float()) / torch.tensor(15.0)).clamp_min(0).bfloat16()
    s = scale.float().unsqueeze(-1)
    n = torch.where(s > 0, torch.round((x - bias.float().unsqueeze(-1)) / s).clamp(0, 15), torch.zeros_like(x))
    n = n.nan_to_num(0).to(torch.uint8).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), torch.stack((scale, bias), -1)


def values(codes, scales):
    """64-bit rows that codes and scales stand for."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double().unflatten(-1, (-1, 64))
    s = scales.double()
    return (n * s[..., :1] + s[..., 1:]).flatten(-2)


def make_table(lens, page, g, extra=2, width=None):
    need = [-(-n // page) for n in lens]
    pool = sum(need) + extra
    order = torch.randperm(pool, generator=g).int()
    table = torch.full((len(lens), width or max(1, max(need))), -7, dtype=torch.int32)  # unused entries are not read
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table, pool


def poisoned(pool, Hkv, page, D, device="cuda"):
    """A pool whose unwritten places hold NaN scales."""
    c = sdp.cache4_empty(pool, Hkv, D, page, device=device)
    for t in (c.k_codes, c.v_codes):
        t.fill_(0xA5)
    for t in (c.k_scales, c.v_scales):
        t.fill_(math.nan)
    return c


A = 0x10000


def pool_args(**kw):
    a = dict(kc=A, ks=2 * A, vc=3 * A, vs=4 * A, P=8, page=16, table=5 * A, ts=4, mp=4)
    a.update({k: v for k, v in kw.items() if k in a})
    return [a[x] for x in ("kc", "ks", "vc", "vs", "P", "page", "table", "ts", "mp")]


BAD = [
    (dict(D=64), sdp.SDP_ERR_UNSUPPORTED),
    (dict(dtype=3), sdp.SDP_ERR_UNSUPPORTED),
    (dict(page=24), sdp.SDP_ERR_INVALID_ARG),
    (dict(page=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(P=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(mp=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(Hkv=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(nseq=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(tokens=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(ts=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(kc=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(table=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(k=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(cu=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(ks=2 * A + 4), sdp.SDP_ERR_ALIGNMENT),
    (dict(v=A + 8), sdp.SDP_ERR_ALIGNMENT),
    (dict(kst=1020), sdp.SDP_ERR_ALIGNMENT),
    (dict(mp=1 << 28), sdp.SDP_ERR_OVERFLOW),
    (dict(tokens=0, k=0, cu=0), sdp.SDP_OK),
]


@pytest.mark.parametrize("kw,code", BAD)
def test_c_calls_refuse_before_any_launch(kw, code):
    from gqa_flash_attention_gb300 import build, serving
    build.build()
    L = serving._lib()
    a = dict(k=6 * A, kst=1024, v=7 * A, cu=8 * A, lens=9 * A, nseq=2, tokens=5, Hkv=8, D=128, dtype=0)
    a.update({k: v for k, v in kw.items() if k in a})
    rows = [a["k"], a["kst"], 128, a["v"], 1024, 128, a["cu"]]
    tail = [a["nseq"], a["tokens"], a["Hkv"], a["D"], a["dtype"], 0]
    assert L.sdp_cache4_append(*pool_args(**kw), *rows, a["lens"], *tail) == code
    assert L.sdp_cache4_gather(*pool_args(**kw), *rows, *tail) == code
    assert L.sdp_cache4_append(*pool_args(), *rows, 0, *tail) in (sdp.SDP_ERR_INVALID_ARG, code)


def test_binding_refuses():
    with pytest.raises(ValueError):
        sdp.cache4_empty(4, 2, 96, device="cpu")
    with pytest.raises(ValueError):
        sdp.cache4_empty(4, 2, 128, page_size=20, device="cpu")
    c = sdp.cache4_empty(4, 2, 128, 16, device="cpu")
    x = torch.zeros(3, 2, 128, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sdp.cache4_append(c, x, x, i, i[:1], i.view(1, 2))
    with pytest.raises(ValueError):
        sdp.cache4_gather(c, i, i.view(1, 2), 3)


CASES = []
for dt in ("fp16", "bf16"):
    CASES += [
        ([1], [1], 1, 128, 16, dt),
        ([17, 1, 40, 33], [17, 1, 3, 1], 8, 128, 16, dt),
        ([100, 5, 300], [0, 5, 171], 2, 256, 64, dt),
        ([50, 49, 48, 47], [2, 49, 1, 0], 3, 128, 48, dt),
        ([260, 7], [260, 7], 1, 256, 256, dt),
        ([31] * 70, [1] * 70, 2, 128, 32, dt),
        ([9] * 1100, [1] * 1100, 1, 256, 16, dt),
        ([2000, 700], [1900, 700], 4, 128, 128, dt),
    ]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new,Hkv,D,page,dt", CASES)
def test_append_then_gather(lens, new, Hkv, D, page, dt):
    g = torch.Generator().manual_seed(len(lens) * 7 + D + page)
    dtype = DTYPES[dt]
    table, pool = make_table(lens, page, g)
    cache = poisoned(pool, Hkv, page, D)
    ref = [t.cpu().clone() for t in cache]
    T = sum(new)
    kv = torch.randn(T, 2 * Hkv, D, generator=g) * torch.exp(3 * torch.randn(T, 1, 1, generator=g))
    kv[:, :, 5] += 4
    if T > 3:
        kv[1] = 0.75            # constant groups
        kv[2] = 0
        kv[3, :, :64] = -2.0    # one constant group beside an ordinary one
    kv = kv.to(dtype).cuda()
    k, v = kv[:, :Hkv], kv[:, Hkv:]  # strided rows
    cu_new = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32)
    dlens, dtable = torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda()
    # rows behind the last sequence are left out: two more rows of input
    pad = torch.cat((kv, torch.full((2, 2 * Hkv, D), math.inf, dtype=dtype, device="cuda")))
    sdp.cache4_append(cache, pad[:, :Hkv], pad[:, Hkv:], cu_new.cuda(), dlens, dtable)
    assert sdp.poll_status() == sdp.SDP_OK
    kq, vq = quantise(k.cpu()), quantise(v.cpu())
    for s, (n, m) in enumerate(zip(lens, new)):
        for i in range(m):
            t = n - m + i
            at, off, r = table[s, t // page], t % page, cu_new[s] + i
            for x, y in zip(ref, (kq[0], kq[1], vq[0], vq[1])):
                x[at, :, off] = y[r]
    for got, want in zip(cache, ref):
        got = got.cpu()
        if got.dtype == torch.bfloat16:
            got, want = got.view(torch.int16), want.view(torch.int16)
        assert torch.equal(got, want)

    # gather the written tails' sequences whole where they are whole, with guard rows around
    full = [n if n == m else 0 for n, m in zip(lens, new)]
    total = sum(full)
    cu = torch.tensor([0] + torch.tensor(full).cumsum(0).tolist(), dtype=torch.int32)
    buf = torch.full((total + 3, 2 * Hkv, D), 7.0, dtype=dtype, device="cuda")
    ko, vo = sdp.cache4_gather(cache, cu.cuda(), dtable, total + 3, dtype=dtype, k_out=buf[:, :Hkv], v_out=buf[:, Hkv:])
    assert sdp.poll_status() == sdp.SDP_OK
    assert (buf[total:] == 7).all()
    for s, n in enumerate(full):
        if n:
            rows = torch.arange(n)
            at, off = table[s, rows // page].long(), rows % page
            for got, c, sc in ((ko, ref[0], ref[1]), (vo, ref[2], ref[3])):
                want = values(c[at, :, off], sc[at, :, off])
                x = got[cu[s]:cu[s] + n].double().cpu()
                tol = (torch.finfo(dtype).eps / 2 + 2.0 ** -24) * want.abs() + 2.0 ** -25
                # fp16 inputs past the type's range are infinities: their groups read NaN (0 * inf)
                nan = torch.isnan(want)
                assert torch.equal(torch.isnan(x), nan)
                bad = ((x - want).abs() > tol) & ~nan
                assert not bad.any(), (int(bad.sum()), x[bad][:3], want[bad][:3])


@pytest.mark.gpu
def test_values_at_their_limits():
    """Largest values, subnormals, infinities and NaN: the group that holds them, and no other."""
    x = torch.randn(6, 1, 128).to(torch.bfloat16)
    big = torch.finfo(torch.bfloat16).max
    x[0, 0, 3], x[0, 0, 9] = big / 4, -big / 4
    x[1, 0, :64] = torch.linspace(0, 1e-39, 64).to(torch.bfloat16)  # subnormal steps
    x[2, 0, 70] = math.inf
    x[3, 0, 70] = math.nan
    x[4, 0, 70] = -math.inf
    cache = sdp.cache4_empty(1, 1, 128, 16)
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    sdp.cache4_append(cache, x.cuda(), x.cuda(), i(0, 6), i(6), i(0).view(1, 1))
    k, v = sdp.cache4_gather(cache, i(0, 6), i(0).view(1, 1), 6, dtype=torch.bfloat16)
    assert sdp.poll_status() == sdp.SDP_OK
    assert torch.equal(k.view(torch.int16), v.view(torch.int16))
    k = k.cpu()
    c, s = quantise(x[[0, 1, 5]])
    want = values(c, s)
    assert ((k[[0, 1, 5]].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -24) * want.abs() + 1e-40).all()
    for r in (2, 3, 4):
        assert torch.isfinite(k[r, 0, :64]).all() and torch.isnan(k[r, 0, 64:]).all()


@pytest.mark.gpu
def test_bad_offsets_lengths_and_pages_are_skipped_and_reported():
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(4, 2, 128, device="cuda").half()

    def run(cu, lens, table, code):
        cache = poisoned(4, 2, 16, 128)
        before = [t.clone() for t in cache]
        sdp.cache4_append(cache, x, x, cu, lens, table)
        assert sdp.poll_status() == code
        return cache, before

    same = lambda a, b: all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))  # noqa: E731
    one = i(0).view(1, 1)
    assert same(*run(i(0, 5), i(5), one, sdp.SDP_ERR_BAD_SEQLENS))       # offsets past the rows
    assert same(*run(i(-1, 4), i(5), one, sdp.SDP_ERR_BAD_SEQLENS))
    assert same(*run(i(0, 4), i(3), one, sdp.SDP_ERR_BAD_SEQLENS))       # shorter than its new rows
    assert same(*run(i(0, 4), i(2 ** 31 - 1), one, sdp.SDP_ERR_BAD_SEQLENS))
    assert same(*run(i(0, 4), i(4), i(4).view(1, 1), sdp.SDP_ERR_BAD_PAGES))
    assert same(*run(i(0, 4), i(4), i(-1).view(1, 1), sdp.SDP_ERR_BAD_PAGES))
    # one bad sequence leaves the others whole; rows past the table's width are skipped
    cache, before = run(i(0, 2, 4), i(2, 17), i(1, 2).view(2, 1), sdp.SDP_ERR_BAD_SEQLENS)
    assert torch.isfinite(cache.k_scales[1, :, :2].float()).all()
    assert torch.isnan(cache.k_scales[1, :, 2:].float()).all()
    run(i(0, 3, 1, 4), i(3, 1, 3), i(0, 1, 2).view(3, 1), sdp.SDP_ERR_BAD_SEQLENS)  # offsets that go down
    out = torch.full((4, 2, 128), 3.0, device="cuda", dtype=torch.half)
    sdp.cache4_gather(cache, i(0, 4), i(9).view(1, 1), 4, dtype=torch.half, k_out=out, v_out=out.clone())
    assert sdp.poll_status() == sdp.SDP_ERR_BAD_PAGES and (out == 3).all()


@pytest.mark.gpu
def test_graph_stream_and_binding_checks():
    g = torch.Generator().manual_seed(2)
    lens = [20, 33]
    table, pool = make_table(lens, 16, g, width=4)
    table = table.clamp_min(0).cuda()
    cache = sdp.cache4_empty(pool, 2, 128, 16)
    k, v = (torch.randn(2, 2, 128, device="cuda").bfloat16() for _ in range(2))
    cu, dl = torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    out = [torch.zeros(2, 2, 128, device="cuda").bfloat16() for _ in range(2)]
    sdp.cache4_append(cache, k, v, cu, dl, table)  # the first call allocates the status word
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdp.cache4_append(cache, k, v, cu, dl, table)
    for step in range(3):  # a decode loop: one more token each, the same graph
        k.copy_(torch.randn(2, 2, 128, device="cuda"))
        graph.replay()
        for s in range(2):
            t = lens[s] + step - 1
            at = table[s, t // 16].item()
            c, sc = quantise(k[s].cpu())
            assert torch.equal(cache.k_codes[at, :, t % 16].cpu(), c)
            assert torch.equal(cache.k_scales[at, :, t % 16].cpu(), sc)
        dl += 1
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ref = sdp.cache4_gather(cache, cu, table, 2)
    sdp.cache4_gather(cache, cu, table, 2, k_out=out[0], v_out=out[1], stream=st)
    st.synchronize()
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    assert sdp.poll_status() == sdp.SDP_OK
    ok = dict(cache=cache, k=k, v=v, cu_seqlens=cu, cache_lens=dl, block_table=table)
    for kw in (dict(k=k.float()), dict(k=k[:, :1]), dict(v=v[:1]), dict(cu_seqlens=cu[:2]), dict(cache_lens=dl.long()),
               dict(block_table=table.t()), dict(block_table=table.cpu()), dict(k=k.cpu(), v=v.cpu()),
               dict(cache=cache._replace(k_scales=cache.k_scales.half())),
               dict(cache=cache._replace(v_codes=cache.v_codes[:1])), dict(k=k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            sdp.cache4_append(**{**ok, **kw})
    with pytest.raises(ValueError):
        sdp.cache4_gather(cache, cu, table, 2, dtype=torch.float32)
    with pytest.raises(ValueError):
        sdp.cache4_append(**{**ok, "k": k.clone().requires_grad_()})
