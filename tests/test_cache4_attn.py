"""Attention over the 4-bit paged cache (sdp_fwd_cache4): refusals on the CPU; on the GPU every row
against the definition in 64 bits on the very codes and scales.

Tolerance, for a column with queries q and keys and values of scales sk, sv and values v: a score
is the sum over groups of s * sum q n + b * sum q with n in 0..15, its products exact (11 bits by
four, the row of q times a power of two; channels below 2^-25 of the largest are off by 2^-36 of it
at most), accumulated in fp32 by the tensor core (each step may drop a bit of the running sum's last
place, 2^-23 of it; D / 16 steps a group and two more): its error is at most
e = scale * sum_c |q_c| * max sk * 16 * 2^-19 + 2^-22 * |score| (scale, ex2 argument). Weights are
then off by a factor 1 + 2 e at most, the stored value by
    finfo.eps / 2 * |o|  (half a step)  +  2 e * max |v|
    + 15 max |sv| * (2^-11 for bf16: weights times scales in one fp16, half a step; 2^-21 for fp16: in
      two)  +  15 max |sv| * 2^-14  (O's steps: at most 5120 / 16 here, 2^-23 each; with 2^-21 less
      than 2^-14)  +  n keys * 15 * 2 max |sv| * 2^-31  (weights times scales among fp16's subnormals,
      2^-25 of 64 for 2 max |sv|)  +  2^-25 (fp16 subnormals of the output),
the log-sum-exp by e + 2^-20 * (1 + |lse|).
"""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp
from test_cache4 import make_table, quantise, values

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
A = 0x10000


def c_call(**kw):
    from gqa_flash_attention_gb300 import serving
    a = dict(q=A, kc=2 * A, ks=3 * A, vc=4 * A, vs=5 * A, P=8, page=16, table=6 * A, ts=4, mp=4, lens=7 * A, o=8 * A,
             lse=9 * A, nseq=2, rows=1, Hq=8, Hkv=2, D=128, scale=0.1, dtype=0, window=0, sinks=0, ws=10 * A, wb=1 << 30)
    a.update(kw)
    return serving._lib().sdp_fwd_cache4(*a.values(), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(D=192), sdp.SDP_ERR_UNSUPPORTED),
    (dict(dtype=2), sdp.SDP_ERR_UNSUPPORTED),
    (dict(rows=33), sdp.SDP_ERR_UNSUPPORTED),
    (dict(rows=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(nseq=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(Hq=7), sdp.SDP_ERR_INVALID_ARG),
    (dict(page=8), sdp.SDP_ERR_INVALID_ARG),
    (dict(P=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(mp=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(window=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(sinks=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(scale=math.nan), sdp.SDP_ERR_INVALID_ARG),
    (dict(q=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(vs=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(ws=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(o=A), sdp.SDP_ERR_INVALID_ARG),
    (dict(kc=2 * A + 8), sdp.SDP_ERR_ALIGNMENT),
    (dict(lse=9 * A + 2), sdp.SDP_ERR_ALIGNMENT),
    (dict(ws=10 * A + 4), sdp.SDP_ERR_ALIGNMENT),
    (dict(mp=1 << 27), sdp.SDP_ERR_OVERFLOW),
    (dict(nseq=1 << 20, Hkv=1 << 12, Hq=1 << 12), sdp.SDP_ERR_OVERFLOW),
])
def test_c_call_refuses_before_any_launch(kw, code):
    from gqa_flash_attention_gb300 import build, serving
    build.build()
    assert c_call(**kw) == code
    if code != sdp.SDP_ERR_ALIGNMENT and set(kw) <= {"D", "dtype", "rows", "nseq", "Hq", "Hkv"}:
        a = dict(nseq=2, rows=1, Hq=8, Hkv=2, D=128, dtype=0)
        a.update(kw)
        assert serving._lib().sdp_fwd_cache4_workspace_bytes(*[a[x] for x in ("nseq", "rows", "Hq", "Hkv", "D", "dtype")]) == code


# ------------------------------------------------------------------ GPU


def fill(lens, Hkv, D, page, dtype, g, kscale=1.0):
    """A pool with the sequences' rows in it and NaN scales everywhere else, and its 64-bit rows."""
    table, pool = make_table(lens, page, g)
    cache = sdp.cache4_empty(pool, Hkv, D, page, device="cpu")
    for t in (cache.k_codes, cache.v_codes):
        t.fill_(0x5A)
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(math.nan)
    ks, vs = [], []
    for s, n in enumerate(lens):
        k = kscale * torch.randn(n, Hkv, D, generator=g)
        k[:, :, 7] += 3
        v = torch.randn(n, Hkv, D, generator=g) * torch.exp(torch.randn(n, 1, 1, generator=g)) + 0.3
        (kc, ksc), (vc, vsc) = quantise(k.to(dtype)), quantise(v.to(dtype))
        t = torch.arange(n)
        at, off = table[s, t // page].long(), t % page
        cache.k_codes[at, :, off], cache.k_scales[at, :, off] = kc, ksc
        cache.v_codes[at, :, off], cache.v_scales[at, :, off] = vc, vsc
        ks.append((values(kc, ksc), ksc[..., 0].double().abs()))
        vs.append((values(vc, vsc), vsc[..., 0].double().abs()))
    return sdp.Cache4(*(t.cuda() for t in cache)), table, ks, vs


def reference(q, k, v, pos, scale, window, sinks):
    """q [rows, Hq, D]; k, v [n, Hkv, D] (64 bits): o, lse."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    j = torch.arange(k.shape[0])
    seen = j[None] <= pos[:, None]
    if window:
        seen &= (j[None] > pos[:, None] - window) | (j[None] < sinks)
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("nhd,jhd->nhj", q.double(), kk) * scale
    s = s.masked_fill(~seen[:, None], -math.inf)
    lse = torch.logsumexp(s, -1) if k.shape[0] else torch.full((n, Hq), -math.inf, dtype=torch.float64)
    w = torch.exp(s - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[..., None])
    return torch.einsum("nhj,jhd->nhd", w, vv), lse


def check(q, o, lse, lens, ks, vs, dtype, window=0, sinks=0, scale=None):
    rows, D = q.shape[1], q.shape[3]
    scale = 1 / math.sqrt(D) if scale is None else scale
    o, lse, q = o.double().cpu(), None if lse is None else lse.double().cpu(), q.cpu()
    W = 15 * (2.0 ** -11 + 2.0 ** -14 if dtype == torch.bfloat16 else 2.0 ** -14)
    for s, n in enumerate(lens):
        pos = torch.arange(n - rows, n)
        ro, rl = reference(q[s], ks[s][0], vs[s][0], pos, scale, window, sinks)
        none = rl.isinf()
        assert (o[s][none] == 0).all()
        if lse is not None:
            assert torch.equal(lse[s][none], rl[none])
        if n == 0:
            continue
        top = rl.masked_fill(none, 0).abs()
        e = abs(scale) * q[s].double().abs().sum(-1) * ks[s][1].max() * 16 * 2.0 ** -19 + 2.0 ** -22 * (top + 20)
        tol = (torch.finfo(dtype).eps / 2 * ro.abs() + 2 * e[..., None] * vs[s][0].abs().max()
               + vs[s][1].max() * (W + n * 15 * 2.0 ** -30) + 2.0 ** -25)
        bad = ((o[s] - ro).abs() > tol) | torch.isnan(o[s])
        assert not bad.any(), (s, n, int(bad.sum()), (o[s] - ro).abs()[bad].max(), tol[bad].max())
        if lse is not None:
            off = ((lse[s] - rl).abs() > e + 2.0 ** -20 * (1 + top))[~none]
            assert not off.any(), (s, n, (lse[s] - rl).abs()[~none].max())


CASES = []
for dt in ("fp16", "bf16"):
    CASES += [
        # lens, rows, Hq, Hkv, D, page, window, sinks
        ([1], 1, 1, 1, 128, 16, 0, 0, dt),
        ([31, 32, 33, 0, 64], 1, 8, 2, 128, 16, 0, 0, dt),
        ([500], 1, 32, 8, 128, 16, 0, 0, dt),
        ([77, 0, 0, 1300], 1, 16, 1, 256, 64, 0, 0, dt),
        ([200, 9], 1, 7, 1, 256, 48, 0, 0, dt),
        ([1000, 17, 333], 1, 8, 8, 128, 32, 0, 0, dt),        # multi-head
        ([700, 40, 2], 4, 8, 2, 128, 128, 0, 0, dt),          # rows, one sequence shorter than them
        ([90, 300], 5, 14, 2, 256, 16, 0, 0, dt),             # 35 columns: three chunks
        ([100, 400], 1, 40, 2, 128, 16, 0, 0, dt),            # 20 heads a group: two chunks
        ([5000, 30, 31, 1], 1, 4, 2, 128, 256, 64, 4, dt),
        ([2000, 257, 64, 65], 3, 8, 2, 128, 16, 50, 33, dt),
        ([600, 12], 1, 4, 4, 256, 64, 1, 0, dt),              # window of one: its own key
        ([600, 12], 2, 4, 4, 256, 64, 1, 1, dt),
        ([300], 1, 4, 1, 128, 32, 100, 1000, dt),             # more sinks than keys
        ([300], 1, 4, 1, 128, 32, 100000, 3, dt),             # a window longer than the sequence
    ]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,rows,Hq,Hkv,D,page,window,sinks,dt", CASES)
def test_every_row(lens, rows, Hq, Hkv, D, page, window, sinks, dt):
    g = torch.Generator().manual_seed(sum(lens) + rows + D)
    dtype = DTYPES[dt]
    cache, table, ks, vs = fill(lens, Hkv, D, page, dtype, g)
    q = torch.randn(len(lens), rows, Hq, D, generator=g).to(dtype).cuda()
    dl, dt_ = torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda()
    n = q.numel()
    obuf = torch.full((n + 512,), math.nan, dtype=dtype, device="cuda")
    lbuf = torch.full((n // D + 64,), math.nan, device="cuda")
    need = sdp.cache4_workspace_bytes(len(lens), rows, Hq, Hkv, D, dtype)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    o, lse = obuf[:n].view(q.shape), lbuf[:n // D].view(q.shape[:-1])
    sdp.fwd_cache4(q, cache, dl, dt_, window=window, sinks=sinks, out=o, lse=lse, workspace=ws[:need])
    assert sdp.poll_status() == sdp.SDP_OK
    assert torch.isnan(obuf[n:]).all() and torch.isnan(lbuf[n // D:]).all() and (ws[need:] == 255).all()
    check(q, o, lse, lens, ks, vs, dtype, window, sinks)
    # the same bits again, without a workspace or a log-sum-exp of the caller's
    o2, l2 = sdp.fwd_cache4(q, cache, dl, dt_, window=window, sinks=sinks)
    assert torch.equal(o2, o) and torch.equal(l2, lse)
    o3, none = sdp.fwd_cache4(q, cache, dl, dt_, window=window, sinks=sinks, return_lse=False)
    assert torch.equal(o3, o) and none is None
    if rows == 1:
        o4, l4 = sdp.fwd_cache4(q[:, 0], cache, dl, dt_, window=window, sinks=sinks)
        assert torch.equal(o4, o[:, 0]) and torch.equal(l4, lse[:, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("nseq", [150, 257, 700])
def test_many_sequences(nseq):
    """More sequences than a block has threads, and than there are CTAs; lengths of zero among them."""
    g = torch.Generator().manual_seed(nseq)
    lens = torch.randint(0, 70, (nseq,), generator=g).tolist()
    cache, table, ks, vs = fill(lens, 2, 128, 16, torch.bfloat16, g)
    q = torch.randn(nseq, 1, 4, 128, generator=g).bfloat16().cuda()
    o, lse = sdp.fwd_cache4(q, cache, torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda())
    assert sdp.poll_status() == sdp.SDP_OK
    check(q, o, lse, lens, ks, vs, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dt,rows", [(256, "fp16", 1), (128, "bf16", 2)])
def test_many_problems_of_many_columns(D, dt, rows):
    """Joins of a column a warp, more columns than a block has warps, one long sequence among short and empty
    ones; a bad length in their midst leaves its own rows alone."""
    g = torch.Generator().manual_seed(D)
    dtype, Hq, Hkv = DTYPES[dt], 40, 2
    lens = torch.randint(0, 90, (170,), generator=g).tolist()
    lens[33], lens[100:103] = 2100, [0, 0, 1]
    cache, table, ks, vs = fill(lens, Hkv, D, 16, dtype, g)
    q = torch.randn(len(lens), rows, Hq, D, generator=g).to(dtype).cuda()
    dl = torch.tensor(lens, dtype=torch.int32)
    ws = torch.full((sdp.cache4_workspace_bytes(len(lens), rows, Hq, Hkv, D, dtype),), 255, dtype=torch.uint8, device="cuda")
    o, lse = sdp.fwd_cache4(q, cache, dl.cuda(), table.cuda(), workspace=ws)
    assert sdp.poll_status() == sdp.SDP_OK
    check(q, o, lse, lens, ks, vs, dtype)
    dl[50] = -3
    o2 = torch.full_like(o, 9)
    _, lse2 = sdp.fwd_cache4(q, cache, dl.cuda(), table.cuda(), out=o2, workspace=ws)
    assert sdp.poll_status() == sdp.SDP_ERR_BAD_SEQLENS
    assert (o2[50] == 9).all()
    keep = [i for i in range(len(lens)) if i != 50]
    check(q[keep], o2[keep], lse2[keep], [lens[i] for i in keep], [ks[i] for i in keep], [vs[i] for i in keep], dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_scales_and_loud_keys(scale, dt):
    g = torch.Generator().manual_seed(8)
    dtype = DTYPES[dt]
    lens = [900, 35]
    cache, table, ks, vs = fill(lens, 2, 128, 32, dtype, g, kscale=4.0)
    q = (2 * torch.randn(2, 1, 8, 128, generator=g)).to(dtype).cuda()
    o, lse = sdp.fwd_cache4(q, cache, torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), scale=scale)
    assert sdp.poll_status() == sdp.SDP_OK
    check(q, o, lse, lens, ks, vs, dtype, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_scales_of_every_size(dt):
    """Scales of V that grow, shrink, are 0, are below it (no quantiser gives one) and, in bf16, near the ends of
    the range; rows of q of very different sizes."""
    g = torch.Generator().manual_seed(21)
    dtype, lens = DTYPES[dt], [700, 700, 90, 64]
    cache, table, ks, vs = fill(lens, 1, 128, 16, dtype, g)
    for s, n in enumerate(lens):
        t = torch.arange(n)
        sc = torch.rand(n, 2, generator=g) + 0.1
        if s == 0:
            sc = sc * 2.0 ** (t[:, None] / 50)
        elif s == 1:
            sc = sc * 2.0 ** (-t[:, None] / 20)
        elif s == 2:
            sc[t % 3 == 0] *= -4
        else:
            sc = torch.zeros_like(sc)
        if dt == "bf16" and s < 2:
            sc = sc * 2.0 ** (110 if s == 0 else -110)
        at, off = table[s, t // 16].long().cuda(), (t % 16).cuda()
        scales = cache.v_scales[at, 0, off].cpu()  # [n, 2 groups, (scale, bias)]
        scales[..., 0] = sc.bfloat16()
        cache.v_scales[at, 0, off] = scales.cuda()
        codes = cache.v_codes[at, 0, off].cpu()
        vs[s] = (values(codes, scales)[:, None], scales[..., 0].double().abs()[:, None])
    q = torch.randn(4, 3, 4, 128, generator=g)
    q[:, 1] *= 1e-4
    q[:, 2, 1:3] *= torch.tensor([3e-8, 40.0])[:, None]
    q = q.to(dtype).cuda()
    o, lse = sdp.fwd_cache4(q, cache, torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda())
    assert sdp.poll_status() == sdp.SDP_OK
    keep = [0, 1, 2, 3] if dt == "bf16" else [1, 2, 3]  # 15 * 2^14 and its sums are near fp16's end
    check(q[keep], o[keep], lse[keep], [lens[i] for i in keep], [ks[i] for i in keep], [vs[i] for i in keep], dtype)


@pytest.mark.gpu
def test_nan_and_infinity_outside_the_window_stay_there():
    g = torch.Generator().manual_seed(5)
    lens, window, sinks = [400], 64, 4
    cache, table, ks, vs = fill(lens, 1, 128, 16, torch.bfloat16, g)
    t = torch.arange(sinks, 400 - window)  # in the sequence, seen by no row
    at, off = table[0, t // 16].long().cuda(), (t % 16).cuda()
    cache.k_scales[at, :, off] = math.nan
    cache.v_scales[at, :, off] = math.inf
    q = torch.randn(1, 1, 4, 128, generator=g).bfloat16().cuda()
    o, lse = sdp.fwd_cache4(q, cache, torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), window=window, sinks=sinks)
    check(q, o, lse, lens, ks, vs, torch.bfloat16, window, sinks)
    cache.v_scales[table[0, 399 // 16], 0, 399 % 16, 1] = math.nan  # a key that is seen: two groups, one of them
    o, _ = sdp.fwd_cache4(q, cache, torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), window=window, sinks=sinks)
    assert torch.isnan(o[..., 64:]).all() and torch.isfinite(o[..., :64]).all()
    # queries that hold a NaN give NaN rows, the others of the same tile not
    q[0, 0, 2, 5] = math.nan
    o, lse = sdp.fwd_cache4(q, cache, torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda(), window=window, sinks=sinks)
    assert torch.isnan(o[0, 0, 2]).all() and torch.isnan(lse[0, 0, 2]) and torch.isfinite(o[0, 0, 1, :64]).all()


@pytest.mark.gpu
def test_bad_lengths_and_pages_are_reported():
    g = torch.Generator().manual_seed(6)
    lens = [50, 40, 60]
    cache, table, ks, vs = fill(lens, 2, 128, 16, torch.float16, g)
    q = torch.randn(3, 1, 4, 128, generator=g).half().cuda()
    for bad in (-1, 65, 2 ** 31 - 1):  # the table holds 4 pages of 16
        dl = torch.tensor([50, bad, 60], dtype=torch.int32).cuda()
        o = torch.full_like(q, 9)
        _, lse = sdp.fwd_cache4(q, cache, dl, table.cuda(), out=o)
        assert sdp.poll_status() == sdp.SDP_ERR_BAD_SEQLENS
        assert (o[1] == 9).all()
        check(q[[0, 2]], o[[0, 2]], lse[[0, 2]], [50, 60], [ks[0], ks[2]], [vs[0], vs[2]], torch.float16)
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    for bad in (-1, 10 ** 6):
        t = table.clone()
        t[1, 1] = bad
        o, lse = sdp.fwd_cache4(q, cache, dl, t.cuda())
        assert sdp.poll_status() == sdp.SDP_ERR_BAD_PAGES
        check(q[[0, 2]], o[[0, 2]], lse[[0, 2]], [50, 60], [ks[0], ks[2]], [vs[0], vs[2]], torch.float16)


@pytest.mark.gpu
def test_waits_that_run_out_are_reported():
    g = torch.Generator().manual_seed(6)
    cache, table, ks, vs = fill([300], 2, 128, 16, torch.float16, g)
    q = torch.randn(1, 1, 4, 128, generator=g).half().cuda()
    dl, t = torch.tensor([300], dtype=torch.int32).cuda(), table.cuda()
    old_ms, old = sdp.set_wait_timeout_ms(50), sdp.set_debug_flags(1)
    try:
        sdp.fwd_cache4(q, cache, dl, t)
        assert sdp.poll_status() == sdp.SDP_ERR_DEVICE_TIMEOUT
        assert sdp.last_status_detail() & 0xff == 3
    finally:
        sdp.set_wait_timeout_ms(old_ms)
        sdp.set_debug_flags(old)
    o, lse = sdp.fwd_cache4(q, cache, dl, t)
    assert sdp.poll_status() == sdp.SDP_OK
    check(q, o, lse, [300], ks, vs, torch.float16)


@pytest.mark.gpu
def test_a_captured_step_follows_lengths_and_pages():
    """One graph serves a decode loop: append a token, attend; lengths grow on the device."""
    g = torch.Generator().manual_seed(12)
    dtype, D, Hkv, Hq = torch.bfloat16, 128, 2, 8
    lens, steps, page = [30, 0, 95], 40, 16
    table, pool = make_table([n + steps for n in lens], page, g)
    cache = sdp.cache4_empty(pool, Hkv, D, page)
    hist = torch.randn(3, max(lens) + steps, 2 * Hkv, D, generator=g).to(dtype)
    dt_ = table.cuda()
    cu = torch.tensor([0, 30, 30, 125], dtype=torch.int32).cuda()
    pre = torch.cat([hist[s, :n] for s, n in enumerate(lens)]).cuda()
    dl = torch.tensor(lens, dtype=torch.int32).cuda()
    sdp.cache4_append(cache, pre[:, :Hkv], pre[:, Hkv:], cu, dl, dt_)
    q, kv = torch.zeros(3, Hq, D, dtype=dtype).cuda(), torch.zeros(3, 2 * Hkv, D, dtype=dtype).cuda()
    one = torch.arange(4, dtype=torch.int32).cuda()
    o, lse = torch.zeros_like(q), torch.zeros(3, Hq).cuda()
    ws = torch.empty(sdp.cache4_workspace_bytes(3, 1, Hq, Hkv, D, dtype), dtype=torch.uint8, device="cuda")
    sdp.fwd_cache4(q, cache, dl, dt_, out=o, lse=lse, workspace=ws)  # set-up outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dl += 1
        sdp.cache4_append(cache, kv[:, :Hkv], kv[:, Hkv:], one, dl, dt_)
        sdp.fwd_cache4(q, cache, dl, dt_, window=48, sinks=2, out=o, lse=lse, workspace=ws)
    for step in range(steps):
        now = [n + step for n in lens]
        q.copy_(torch.randn(3, Hq, D, generator=g))
        kv.copy_(torch.stack([hist[s, now[s]] for s in range(3)]))
        graph.replay()
        if step % 13 and step != steps - 1:
            continue
        ks, vs = [], []
        for s in range(3):
            for out, h in ((ks, hist[s, :now[s] + 1, :Hkv]), (vs, hist[s, :now[s] + 1, Hkv:])):
                c, sc = quantise(h)
                out.append((values(c, sc), sc[..., 0].double().abs()))
        check(q[:, None], o[:, None], lse[:, None], [n + 1 for n in now], ks, vs, dtype, 48, 2)
    assert sdp.poll_status() == sdp.SDP_OK


@pytest.mark.gpu
def test_two_graphs_at_once_with_a_workspace_each():
    """Their joins start beside the attention of either; a following call in the graph reads what they wrote."""
    g = torch.Generator().manual_seed(16)
    lens = [[1500, 40, 0], [700, 900, 5]]
    graphs, res, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for ln in lens:
        cache, table, ks, vs = fill(ln, 2, 128, 32, torch.bfloat16, g)
        q = torch.randn(3, 1, 8, 128, generator=g).bfloat16().cuda()
        dl, t = torch.tensor(ln, dtype=torch.int32).cuda(), table.cuda()
        ws = torch.empty(sdp.cache4_workspace_bytes(3, 1, 8, 2, 128, torch.bfloat16), dtype=torch.uint8, device="cuda")
        o, lse, copy = torch.zeros_like(q), torch.zeros(3, 1, 8).cuda(), torch.zeros_like(q)
        sdp.fwd_cache4(q, cache, dl, t, out=o, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                sdp.fwd_cache4(q, cache, dl, t, out=o, lse=lse, workspace=ws)
                copy.copy_(o)
                o.zero_()
        graphs.append(graph)
        res.append((q, copy, lse, ln, ks, vs, (cache, dl, t, ws, o)))
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for q, o, lse, ln, ks, vs, _ in res:
        check(q, o, lse, ln, ks, vs, torch.bfloat16)
    assert sdp.poll_status() == sdp.SDP_OK


@pytest.mark.gpu
def test_two_streams_at_once_and_binding_checks():
    g = torch.Generator().manual_seed(15)
    lens = [3000, 1500, 64]
    cache, table, ks, vs = fill(lens, 2, 256, 64, torch.float16, g)
    q = torch.randn(3, 1, 16, 256, generator=g).half().cuda()
    dl, t = torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda()
    want, lwant = sdp.fwd_cache4(q, cache, dl, t)
    check(q, want, lwant, lens, ks, vs, torch.float16)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[sdp.fwd_cache4(q, cache, dl, t, stream=s) for s in streams] for _ in range(8)]
    torch.cuda.synchronize()
    for row in got:
        for o, l in row:
            assert torch.equal(o, want) and torch.equal(l, lwant)
    o, _ = sdp.fwd_cache4(q, cache, dl, t, stream=streams[0].cuda_stream)  # a raw handle
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    assert sdp.poll_status() == sdp.SDP_OK
    ok = dict(q=q, cache=cache, cache_lens=dl, block_table=t)
    for kw in (dict(q=q.float()), dict(q=q[0, 0]), dict(q=q[:2]), dict(q=q[..., :128].contiguous()), dict(q=q.cpu()),
               dict(q=q.transpose(0, 2)), dict(cache_lens=dl[:2]), dict(cache_lens=dl.cpu()), dict(block_table=t.long()),
               dict(out=want[:2]), dict(lse=lwant.half()), dict(workspace=torch.empty(8)),
               dict(q=q.clone().requires_grad_()), dict(cache=cache._replace(v_scales=cache.v_scales[:, :1]))):
        with pytest.raises(ValueError):
            sdp.fwd_cache4(**{**ok, **kw})
    for kw in (dict(window=-1), dict(scale=math.nan), dict(workspace=torch.empty(64, device="cuda")),
               dict(q=q[:, :, :15].contiguous())):
        with pytest.raises(sdp.SdpError):
            sdp.fwd_cache4(**{**ok, **kw})
    e = sdp.fwd_cache4(q[:0], cache, dl[:0], t[:0])
    assert e[0].shape == (0, 1, 16, 256) and e[1].shape == (0, 1, 16)
