"""Sliding-window attention with first tokens that stay visible (sdp_fwd_window,
sdp_fwd_varlen_window): refusals on the CPU, every row against the definition in 64 bits on the GPU.

Tolerance of an output: half a step of the stored type, finfo.eps / 2 * |o|; the weights rounded to
that type before P V, at most finfo.eps / 2 * sum w |v|; the fp32 scores, which the tensor core sums
D terms of, at most e = 2^-20 * |scale| * max sum |q k| in the exponent and so 2 e * max |v|; 2^-19
* sum w |v| for ex2 and the fp32 sums of a row's at most some thousand weights; and 2^-24 where fp16 is
subnormal. The log-sum-exp: e + 2^-19 * (1 + |lse|).
"""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
A = 0x10000


def dense_call(**kw):
    from gqa_flash_attention_gb300 import serving
    a = dict(q=A, k=2 * A, v=3 * A, o=4 * A, lse=5 * A, B=1, Hq=4, Hkv=2, Sq=300, Skv=300, D=128, scale=0.1, dtype=0,
             window=64, sinks=0)
    a.update(kw)
    return serving._lib().sdp_fwd_window(*a.values(), 0)


def varlen_call(**kw):
    from gqa_flash_attention_gb300 import serving
    a = dict(q=A, k=2 * A, v=3 * A, o=4 * A, lse=5 * A, cu_q=6 * A, cu_k=7 * A, nseq=2, Hq=4, Hkv=2, total_q=300,
             total_k=300, max_q=200, D=128, scale=0.1, dtype=0, window=64, sinks=0)
    a.update(kw)
    return serving._lib().sdp_fwd_varlen_window(*a.values(), 0)


COMMON_BAD = [
    (dict(D=64), sdp.SDP_ERR_UNSUPPORTED),
    (dict(dtype=2), sdp.SDP_ERR_UNSUPPORTED),
    (dict(Hq=5), sdp.SDP_ERR_INVALID_ARG),
    (dict(window=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(window=-4), sdp.SDP_ERR_INVALID_ARG),
    (dict(sinks=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(scale=math.inf), sdp.SDP_ERR_INVALID_ARG),
    (dict(q=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(o=2 * A), sdp.SDP_ERR_INVALID_ARG),
    (dict(v=3 * A + 8), sdp.SDP_ERR_ALIGNMENT),
    (dict(lse=5 * A + 1), sdp.SDP_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,code", COMMON_BAD)
def test_c_calls_refuse_before_any_launch(kw, code):
    from gqa_flash_attention_gb300 import build
    build.build()
    assert dense_call(**kw) == code
    assert varlen_call(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(Sq=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(Skv=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(Skv=1 << 30), sdp.SDP_ERR_OVERFLOW),
    (dict(B=1 << 16, Hq=1 << 16, Hkv=1 << 16), sdp.SDP_ERR_OVERFLOW),
])
def test_dense_call_refuses(kw, code):
    assert dense_call(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(nseq=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(cu_q=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(max_q=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(total_k=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(cu_k=7 * A + 2), sdp.SDP_ERR_ALIGNMENT),
    (dict(nseq=1 << 20, Hq=1 << 12, Hkv=1), sdp.SDP_ERR_OVERFLOW),
    (dict(total_q=0), sdp.SDP_OK),
    (dict(total_q=0, q=0, cu_q=0), sdp.SDP_OK),
])
def test_varlen_call_refuses(kw, code):
    assert varlen_call(**kw) == code


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(1, 2, 8, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        sdp.fwd_window(x, x, x, 4)
    with pytest.raises(ValueError):
        sdp.fwd_varlen_window(x[0], x[0], x[0], torch.zeros(2), torch.zeros(2), 8, 4)


# ------------------------------------------------------------------ GPU


def reference(q, k, v, window, sinks, scale):
    """q [Hq, Sq, D], k and v [Hkv, Skv, D] on the GPU: o, lse, sum w |v|, sum |q k| in 64 bits."""
    G, Sq, Skv = q.shape[0] // k.shape[0], q.shape[1], k.shape[1]
    q, k, v = q.double(), k.double().repeat_interleave(G, 0), v.double().repeat_interleave(G, 0)
    p = torch.arange(Skv - Sq, Skv, device=q.device)[:, None]
    j = torch.arange(Skv, device=q.device)[None]
    seen = (j <= p) & ((j > p - window) | (j < sinks))
    s = (q @ k.transpose(1, 2) * scale).masked_fill(~seen, -math.inf)
    if Skv == 0:
        z = torch.zeros_like(q)
        return z, torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device), z, 0.0
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[..., None])
    w = w.masked_fill(~seen, 0)
    return w @ v, lse, w @ v.abs(), float((q.abs() @ k.abs().transpose(1, 2)).max())


def check(o, lse, q, k, v, window, sinks, scale, dtype):
    """One sequence: o, q [Hq, Sq, D], lse [Hq, Sq] or None."""
    ro, rl, mag, dot = reference(q, k, v, window, sinks, scale)
    eps = torch.finfo(dtype).eps
    none = rl.isinf()
    assert (o[none] == 0).all()
    e = 2.0 ** -20 * abs(scale) * dot
    vmax = float(v.double().abs().max()) if v.numel() else 0.0
    tol = eps / 2 * ro.abs() + (eps / 2 + 2.0 ** -19) * mag + 2 * e * vmax + 2.0 ** -24
    bad = ((o.double() - ro).abs() > tol) | torch.isnan(o)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((o.double() - ro).abs()[bad].max()))
    if lse is not None:
        assert torch.equal(lse.double()[none], rl[none])
        off = ((lse.double() - rl).abs() > e + 2.0 ** -19 * (1 + rl.masked_fill(none, 0).abs()))[~none]
        assert not off.any(), float((lse.double() - rl).abs()[~none].max())


def guarded(shape, dtype, value=math.nan, guard=1024):
    n = math.prod(shape)
    buf = torch.full((n + guard,), value, dtype=dtype, device="cuda")
    return buf[:n].view(shape), buf[n:]


DENSE = []
for dt in ("fp16", "bf16"):
    DENSE += [
        # B, Hq, Hkv, Sq, Skv, D, window, sinks
        (1, 1, 1, 1, 1, 128, 1, 0, dt),
        (1, 4, 1, 256, 256, 128, 64, 4, dt),
        (2, 4, 2, 300, 300, 128, 1, 0, dt),              # a window of one: its own key
        (2, 4, 2, 300, 300, 256, 1, 1, dt),
        (1, 3, 1, 513, 700, 128, 128, 0, dt),            # a chunk behind a prefix; odd group
        (1, 8, 2, 400, 1200, 256, 129, 5, dt),
        (1, 2, 2, 700, 700, 128, 127, 300, dt),          # sinks over several tiles
        (1, 2, 1, 640, 640, 256, 5000, 3, dt),           # a window longer than the sequence: causal
        (1, 2, 2, 900, 200, 128, 100, 7, dt),            # more rows than keys: the first see none
        (3, 8, 2, 1, 1000, 128, 300, 4, dt),             # one row, heads packed
        (1, 16, 1, 5, 2000, 256, 1000, 0, dt),
        (2, 16, 2, 100, 900, 128, 33, 2, dt),            # packed heads over several tiles
        (1, 4, 2, 127, 60, 128, 20, 1, dt),              # packed, rows without keys
        (1, 2, 2, 2500, 2500, 128, 800, 129, dt),
    ]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,Sq,Skv,D,window,sinks,dt", DENSE)
def test_dense_every_row(B, Hq, Hkv, Sq, Skv, D, window, sinks, dt):
    g = torch.Generator(device="cuda").manual_seed(Sq + Skv + window)
    dtype = DTYPES[dt]
    q = torch.randn(B, Hq, Sq, D, device="cuda", generator=g).to(dtype)
    k = (torch.randn(B, Hkv, Skv, D, device="cuda", generator=g) * 1.5).to(dtype)
    v = torch.randn(B, Hkv, Skv, D, device="cuda", generator=g).to(dtype)
    o, og = guarded(q.shape, dtype)
    lse, lg = guarded(q.shape[:3], torch.float32)
    sdp.fwd_window(q, k, v, window, sinks=sinks, out=o, lse=lse)
    assert sdp.poll_status() == sdp.SDP_OK
    assert torch.isnan(og).all() and torch.isnan(lg).all()
    for b in range(B):
        check(o[b], lse[b], q[b], k[b], v[b], window, sinks, 1 / math.sqrt(D), dtype)
    o2, none = sdp.fwd_window(q, k, v, window, sinks=sinks, return_lse=False)
    assert none is None and torch.equal(o2, o)


VARLEN = []
for dt in ("fp16", "bf16"):
    VARLEN += [
        ((1, 127, 128, 129, 300), (1, 127, 128, 129, 300), 4, 2, 128, 64, 2, dt),
        ((0, 40, 0, 200, 7), (10, 0, 0, 150, 33), 8, 2, 256, 30, 4, dt),      # empty, keyless, more rows than keys
        ((50, 257, 3, 140), (500, 257, 900, 1000), 3, 1, 128, 200, 0, dt),    # chunks behind prefixes
        ((1, 1, 1, 1), (1000, 1, 129, 128), 4, 4, 256, 128, 1, dt),           # decoding rows
        ((700,), (1300,), 16, 1, 256, 1, 200, dt),
    ]


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, 32], ids=["compact", "full_grid"])
@pytest.mark.parametrize("lq,lk,Hq,Hkv,D,window,sinks,dt", VARLEN)
def test_varlen_every_row(lq, lk, Hq, Hkv, D, window, sinks, dt, flags):
    g = torch.Generator(device="cuda").manual_seed(sum(lk))
    dtype = DTYPES[dt]
    tq, tk = sum(lq), sum(lk)
    q = torch.randn(tq, Hq, D, device="cuda", generator=g).to(dtype)
    k, v = (torch.randn(tk, Hkv, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    cq, ck = (torch.tensor([0] + torch.tensor(x).cumsum(0).tolist(), dtype=torch.int32).cuda() for x in (lq, lk))
    o, og = guarded(q.shape, dtype)
    lse, lg = guarded((Hq, tq), torch.float32)
    old = sdp.set_debug_flags(flags)
    try:
        sdp.fwd_varlen_window(q, k, v, cq, ck, max(lq), window, sinks=sinks, scale=0.07, out=o, lse=lse)
        assert sdp.poll_status() == sdp.SDP_OK
    finally:
        sdp.set_debug_flags(old)
    assert torch.isnan(og).all() and torch.isnan(lg).all()
    a = b = 0
    for n, m in zip(lq, lk):
        if n:
            check(o[a:a + n].transpose(0, 1), lse[:, a:a + n], q[a:a + n].transpose(0, 1), k[b:b + m].transpose(0, 1),
                  v[b:b + m].transpose(0, 1), window, sinks, 0.07, dtype)
        a, b = a + n, b + m


@pytest.mark.gpu
@pytest.mark.parametrize("nseq", [100, 513])
def test_many_sequences(nseq):
    g = torch.Generator(device="cuda").manual_seed(nseq)
    lens = torch.randint(0, 60, (nseq,), generator=torch.Generator().manual_seed(nseq)).tolist()
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32).cuda()
    q = torch.randn(sum(lens), 2, 128, device="cuda", generator=g).half()
    k, v = (torch.randn(sum(lens), 1, 128, device="cuda", generator=g).half() for _ in range(2))
    o, lse = sdp.fwd_varlen_window(q, k, v, cu, cu, 60, 9, sinks=2)
    assert sdp.poll_status() == sdp.SDP_OK
    a = 0
    for n in lens:
        if n:
            check(*(x.transpose(0, 1) for x in (o[a:a + n],)), lse[:, a:a + n], q[a:a + n].transpose(0, 1),
                  k[a:a + n].transpose(0, 1), v[a:a + n].transpose(0, 1), 9, 2, 1 / math.sqrt(128), torch.float16)
        a += n


@pytest.mark.gpu
def test_one_long_sequence_among_many():
    """The list of tiles that exist against a tile of the longest sequence for every sequence: the same bits."""
    g = torch.Generator().manual_seed(3)
    lq = torch.randint(0, 20, (1100,), generator=g)
    lq[[5, 800]] = torch.tensor([1500, 300])
    lk = lq + torch.randint(0, 9, (1100,), generator=g)
    cu_q, cu_k = (torch.cat((torch.zeros(1, dtype=torch.int64), n.cumsum(0))).int().cuda() for n in (lq, lk))
    q = torch.randn(int(lq.sum()), 8, 128, generator=g).bfloat16().cuda()
    k, v = (torch.randn(int(lk.sum()), 2, 128, generator=g).bfloat16().cuda() for _ in range(2))
    o, lse = sdp.fwd_varlen_window(q, k, v, cu_q, cu_k, 1500, 64, sinks=2)
    old = sdp.set_debug_flags(32)
    try:
        of, lf = sdp.fwd_varlen_window(q, k, v, cu_q, cu_k, 1500, 64, sinks=2)
    finally:
        sdp.set_debug_flags(old)
    assert sdp.poll_status() == sdp.SDP_OK
    assert torch.equal(o, of) and torch.equal(lse, lf) and torch.isfinite(o).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_scales_and_peaks(scale, D):
    """A scale of zero, a negative one, and scores that saturate; maxima that jump between tiles."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(1, 2, 600, D, device="cuda", generator=g).bfloat16()
    k = torch.randn(1, 2, 600, D, device="cuda", generator=g)
    k[:, :, ::97] *= 6
    k = k.bfloat16()
    v = torch.randn(1, 2, 600, D, device="cuda", generator=g).bfloat16()
    o, lse = sdp.fwd_window(q, k, v, 150, sinks=3, scale=scale)
    assert sdp.poll_status() == sdp.SDP_OK
    check(o[0], lse[0], q[0], k[0], v[0], 150, 3, scale, torch.bfloat16)


@pytest.mark.gpu
def test_a_long_window_is_plain_causal_attention():
    g = torch.Generator(device="cuda").manual_seed(4)
    q, k, v = (torch.randn(1, 4, 700, 128, device="cuda", generator=g).half() for _ in range(3))
    o, lse = sdp.fwd_window(q, k, v, 2 ** 31 - 1, sinks=2 ** 31 - 1)
    oc, lc = sdp.sdp_fwd(q, k, v, causal=True)
    assert sdp.poll_status() == sdp.SDP_OK
    # the same function; masked tiles round the scaled score before the maximum is taken off, so not
    # the same bits
    for x, y in ((o, lse), (oc, lc)):
        check(x[0], y[0], q[0], k[0], v[0], 700, 0, 1 / math.sqrt(128), torch.float16)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dt", [(128, "fp16"), (256, "bf16")])
def test_nan_and_infinity_stay_outside_the_window(D, dt):
    """Unseen keys and values that are not finite leave a row alone; seen ones do not."""
    g = torch.Generator(device="cuda").manual_seed(6)
    dtype = DTYPES[dt]
    S, W, sinks = 500, 70, 3
    q, k, v = (torch.randn(1, 2, S, D, device="cuda", generator=g).to(dtype) for _ in range(3))
    clean, lclean = sdp.fwd_window(q, k, v, W, sinks=sinks)
    kb, vb = k.clone(), v.clone()
    kb[0, 0, 200], vb[0, 0, 200, 5] = math.nan, math.inf
    vb[0, 1, 130] = math.nan
    kb[0, 1, 131, 2] = math.inf
    o, lse = sdp.fwd_window(q, kb, vb, W, sinks=sinks)
    assert sdp.poll_status() == sdp.SDP_OK
    for h, bad in ((0, (200,)), (1, (130, 131))):
        hit = torch.zeros(S, dtype=torch.bool, device="cuda")
        for j in bad:
            hit[j:j + W] = True
        kz, vz = k[0, h:h + 1], v[0, h:h + 1]
        # rows that do not see them: as without them, to the tolerance of two roundings of the weights
        ro, rl, mag, dot = reference(q[0, h:h + 1], kz, vz, W, sinks, 1 / math.sqrt(D))
        eps = torch.finfo(dtype).eps
        tol = eps / 2 * ro.abs() + (eps / 2 + 2.0 ** -19) * mag + 2.0 ** -19 * dot + 2.0 ** -24
        off = ((o[0, h:h + 1].double() - ro).abs() > tol) | torch.isnan(o[0, h:h + 1])
        assert not off[:, ~hit].any()
        assert ((lse[0, h:h + 1].double() - rl).abs() < 1e-4)[:, ~hit].all()
    assert torch.isnan(o[0, 0, 200:200 + W]).any(-1).all()
    assert torch.isnan(o[0, 1, 130:130 + W]).all()
    qb = q.clone()
    qb[0, 0, 77, 3] = math.nan  # a query that is not finite: its own row alone
    o, lse = sdp.fwd_window(qb, k, v, W, sinks=sinks)
    assert torch.isnan(o[0, 0, 77]).all() and torch.isnan(lse[0, 0, 77])
    o[0, 0, 77], lse[0, 0, 77] = clean[0, 0, 77], lclean[0, 0, 77]
    assert torch.equal(o, clean) and torch.equal(lse, lclean)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dt", [(128, "bf16"), (256, "fp16")])
@pytest.mark.parametrize("Hq,Hkv,flags", [(8, 2, 0), (8, 2, 2), (9, 3, 0)], ids=["pairs", "single", "odd_group"])
@pytest.mark.parametrize("Sq,Skv", [(150, 100), (300, 300), (129, 700), (300, 5)])
def test_a_large_batch_has_the_bits_of_its_parts(Sq, Skv, D, dt, Hq, Hkv, flags):
    """Several units a CTA, or a pair of CTAs, whose rows a warpgroup of its own writes, against one unit a CTA at
    most; rows without a key, and values that are not finite in and out of sight."""
    g = torch.Generator(device="cuda").manual_seed(Sq + Skv)
    dtype, W, sinks = DTYPES[dt], 40, 3
    B = 20
    q = torch.randn(B, Hq, Sq, D, device="cuda", generator=g).to(dtype)
    k, v = (torch.randn(B, Hkv, Skv, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    v[1, 0, Skv // 2, 3], v[2, 1, 0, 7], k[3, 1, Skv - 1, 0] = math.inf, math.nan, math.nan
    q[4, 5, Sq // 2, 1] = math.nan
    old = sdp.set_debug_flags(flags)
    try:
        o, lse = sdp.fwd_window(q, k, v, W, sinks=sinks)
    finally:
        sdp.set_debug_flags(old)
    for b in range(B):
        ob, lb = sdp.fwd_window(q[b:b + 1], k[b:b + 1], v[b:b + 1], W, sinks=sinks)
        assert torch.equal(ob[0].view(torch.int16), o[b].view(torch.int16)) or torch.equal(
            torch.nan_to_num(ob[0], nan=9), torch.nan_to_num(o[b], nan=9))
        assert torch.equal(torch.nan_to_num(lb[0], nan=9), torch.nan_to_num(lse[b], nan=9))
    # the same rows as a packed batch
    pack = [x.transpose(1, 2).reshape(-1, x.shape[1], D).contiguous() for x in (q, k, v)]
    cu_q, cu_k = (torch.arange(B + 1, dtype=torch.int32, device="cuda") * n for n in (Sq, Skv))
    ov, lv = sdp.fwd_varlen_window(*pack, cu_q, cu_k, Sq, W, sinks=sinks)
    ov, lv = ov.view(B, Sq, Hq, D).transpose(1, 2), lv.view(Hq, B, Sq).transpose(0, 1)
    assert torch.equal(torch.isnan(ov), torch.isnan(o)) and torch.equal(torch.isnan(lv), torch.isnan(lse))
    # (a tile at the end of a sequence also holds the next one's first keys: where those are not finite the rows
    # before them are computed again, in other steps, so bits are compared behind the last such sequence)
    assert torch.equal(torch.nan_to_num(ov[4:], nan=9), torch.nan_to_num(o[4:], nan=9))
    assert torch.equal(torch.nan_to_num(lv[4:], nan=9), torch.nan_to_num(lse[4:], nan=9))
    assert sdp.poll_status() == sdp.SDP_OK
    rows = torch.isnan(o).any(-1)
    assert not rows[[0] + list(range(5, B))].any()
    assert int(rows[4].sum()) == (1 if Skv - Sq + Sq // 2 >= 0 else 0)  # a row without a key is 0, whatever its query
    if Skv < Sq:
        assert (o[:, :, :Sq - Skv][[0] + list(range(5, B))] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
def test_large_batches_in_graphs_on_two_streams(D):
    """Two graphs with several units a CTA, replayed at once with new inputs."""
    g = torch.Generator(device="cuda").manual_seed(D)
    sets = [[torch.randn(6, h, 500, D, device="cuda", generator=g).half() for h in (16, 4, 4)] for _ in range(2)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for q, k, v in sets:
        sdp.fwd_window(q, k, v, 130, sinks=5)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(sdp.fwd_window(q, k, v, 130, sinks=5))
        graphs.append(graph)
    for step in range(3):
        for x in sets:
            for t in x:
                t.copy_(torch.randn(t.shape, device="cuda", generator=g))
        torch.cuda.synchronize()
        for _ in range(4):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for (q, k, v), (o, lse) in zip(sets, outs):
            want, lwant = sdp.fwd_window(q, k, v, 130, sinks=5)
            assert torch.equal(o, want) and torch.equal(lse, lwant)
    assert sdp.poll_status() == sdp.SDP_OK


@pytest.mark.gpu
@pytest.mark.parametrize("D,Hkv", [(128, 32), (256, 4), (256, 32)])
def test_waits_that_run_out_end_a_large_batch(D, Hkv):
    q, k, v = (torch.randn(8, h, 300, D, device="cuda").half() for h in (32, Hkv, Hkv))
    want, lwant = sdp.fwd_window(q, k, v, 70)
    old_ms, old = sdp.set_wait_timeout_ms(20), sdp.set_debug_flags(1)
    try:
        sdp.fwd_window(q, k, v, 70)
        assert sdp.poll_status() == sdp.SDP_ERR_DEVICE_TIMEOUT
    finally:
        sdp.set_wait_timeout_ms(old_ms)
        sdp.set_debug_flags(old)
    o, lse = sdp.fwd_window(q, k, v, 70)
    assert sdp.poll_status() == sdp.SDP_OK and torch.equal(o, want) and torch.equal(lse, lwant)


@pytest.mark.gpu
@pytest.mark.parametrize("flags", [0, 32], ids=["compact", "full_grid"])
def test_bad_offsets_are_reported_and_skipped(flags):
    g = torch.Generator(device="cuda").manual_seed(7)
    q = torch.randn(300, 2, 128, device="cuda", generator=g).half()
    k, v = (torch.randn(300, 1, 128, device="cuda", generator=g).half() for _ in range(2))
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    old = sdp.set_debug_flags(flags)
    try:
        for cq, ck, mx in ((i(0, 100, 301), i(0, 100, 300), 200), (i(0, 100, 300), i(0, 200, 100), 200),
                           (i(-1, 100, 300), i(0, 100, 300), 200), (i(0, 20, 300), i(0, 100, 300), 100)):
            o = torch.full_like(q, 5)
            sdp.fwd_varlen_window(q, k, v, cq, ck, mx, 64, out=o)
            assert sdp.poll_status() == sdp.SDP_ERR_BAD_SEQLENS
            assert (o == 5).any()
        cu = i(0, 100, 300)
        o, lse = sdp.fwd_varlen_window(q, k, v, cu, cu, 200, 64)
        assert sdp.poll_status() == sdp.SDP_OK
        check(o[:100].transpose(0, 1), lse[:, :100], q[:100].transpose(0, 1), k[:100].transpose(0, 1),
              v[:100].transpose(0, 1), 64, 0, 1 / math.sqrt(128), torch.float16)
    finally:
        sdp.set_debug_flags(old)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
def test_waits_that_run_out_are_reported(D):
    q, k, v = (torch.randn(1, 2, 400, D, device="cuda").half() for _ in range(3))
    want, _ = sdp.fwd_window(q, k, v, 100)
    old_ms, old = sdp.set_wait_timeout_ms(50), sdp.set_debug_flags(1)
    try:
        sdp.fwd_window(q, k, v, 100)
        assert sdp.poll_status() == sdp.SDP_ERR_DEVICE_TIMEOUT
        assert 1 <= (sdp.last_status_detail() & 0xff) <= 6
    finally:
        sdp.set_wait_timeout_ms(old_ms)
        sdp.set_debug_flags(old)
    got, _ = sdp.fwd_window(q, k, v, 100)
    assert sdp.poll_status() == sdp.SDP_OK and torch.equal(got, want)


@pytest.mark.gpu
def test_graphs_streams_and_binding_checks():
    g = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn(2, 8, 1000, 128, device="cuda", generator=g).half()
    k, v = (torch.randn(2, 2, 1000, 128, device="cuda", generator=g).half() for _ in range(2))
    want, lwant = sdp.fwd_window(q, k, v, 200, sinks=4)
    o, lse = torch.zeros_like(q), torch.zeros_like(lwant)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdp.fwd_window(q, k, v, 200, sinks=4, out=o, lse=lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graph.replay()
    got = [sdp.fwd_window(q, k, v, 200, sinks=4, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, lwant)
    assert all(torch.equal(a, want) and torch.equal(b, lwant) for a, b in got)
    assert sdp.poll_status() == sdp.SDP_OK
    ok = dict(q=q, k=k, v=v, window=200)
    for kw in (dict(q=q.float()), dict(k=k.bfloat16()), dict(q=q.transpose(1, 2)), dict(v=v[:, :, :9]), dict(k=k.cpu()),
               dict(q=q[0]), dict(out=want[:1]), dict(lse=lwant.half()), dict(q=q.clone().requires_grad_())):
        with pytest.raises(ValueError):
            sdp.fwd_window(**{**ok, **kw})
    for kw in (dict(window=0), dict(sinks=-1), dict(scale=math.nan), dict(q=q[:, :7].contiguous())):
        with pytest.raises(sdp.SdpError):
            sdp.fwd_window(**{**ok, **kw})
    t, u = q[0].transpose(0, 1).contiguous(), k[0].transpose(0, 1).contiguous()
    cu = torch.tensor([0, 1000], dtype=torch.int32, device="cuda")
    ok = dict(q=t, k=u, v=u, cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=1000, window=5)
    for kw in (dict(cu_seqlens_q=cu.long()), dict(cu_seqlens_k=cu[:1]), dict(cu_seqlens_q=cu.cpu()), dict(q=t[0]),
               dict(k=u[:, :, :64].contiguous()), dict(lse=torch.zeros(8, 9, device="cuda"))):
        with pytest.raises(ValueError):
            sdp.fwd_varlen_window(**{**ok, **kw})


@pytest.mark.gpu
def test_a_prompt_in_chunks_over_the_cache():
    """The path as it is used: head norms and rotation, the cache written chunk by chunk, each chunk
    attended over the rows gathered back, then decoding: the same as one window call over the gathered rows."""
    g = torch.Generator(device="cuda").manual_seed(21)
    D, Hq, Hkv, page, W, sinks = 128, 8, 2, 32, 150, 4
    lens = [600, 333]
    T = sum(lens)
    cu = torch.tensor([0, 600, 933], dtype=torch.int32, device="cuda")
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, device="cuda", generator=g).bfloat16()
    q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    w = torch.ones(D, device="cuda", dtype=torch.bfloat16)
    q, k = sdp.qk_norm_rope(q, k, pos, sdp.rope_table(sdp.rope_inv_freq(D, device="cuda")), q_weight=w, k_weight=w)
    pages = [-(-n // page) for n in lens]
    table = torch.zeros(2, max(pages), dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(pages), device="cuda", generator=g).int()
    table[0, :pages[0]], table[1, :pages[1]] = order[:pages[0]], order[pages[0]:]
    cache = sdp.cache4_empty(sum(pages), Hkv, D, page)
    outs = [[], []]
    done = [0, 0]
    for chunk in (200, 1, 130, 600):
        n = [min(chunk, lens[s] - done[s]) for s in range(2)]
        rows = torch.cat([torch.arange(n[s], device="cuda") + int(cu[s]) + done[s] for s in range(2)])
        done = [done[s] + n[s] for s in range(2)]
        cq = torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32, device="cuda")
        dl = torch.tensor(done, dtype=torch.int32, device="cuda")
        sdp.cache4_append(cache, k[rows], v[rows], cq, dl, table)
        ck = torch.tensor([0, done[0], done[0] + done[1]], dtype=torch.int32, device="cuda")
        kg, vg = sdp.cache4_gather(cache, ck, table, sum(done))
        o, _ = sdp.fwd_varlen_window(q[rows], kg, vg, cq, ck, max(max(n), 1), W, sinks=sinks)
        for s in range(2):
            outs[s].append(o[int(cq[s]):int(cq[s + 1])])
    assert done == lens
    kg, vg = sdp.cache4_gather(cache, cu, table, T)
    whole, _ = sdp.fwd_varlen_window(q, kg, vg, cu, cu, 600, W, sinks=sinks)
    assert sdp.poll_status() == sdp.SDP_OK
    got = torch.cat([torch.cat(outs[s]) for s in range(2)])
    for s in range(2):
        r = slice(int(cu[s]), int(cu[s + 1]))
        for x in (whole, got):
            check(x[r].transpose(0, 1), None, q[r].transpose(0, 1), kg[r].transpose(0, 1), vg[r].transpose(0, 1), W, sinks,
                  1 / math.sqrt(D), torch.bfloat16)
    # decoding: the last rows again, straight from the 4-bit cache; its keys and values were rounded to
    # 16 bits by the gather (2^-8 of each: 2^-8 sum |q k| in a score's exponent, 2^-8 sum w |v| in O)
    last = torch.stack([q[int(cu[s + 1]) - 1] for s in range(2)])
    o, _ = sdp.fwd_cache4(last, cache, torch.tensor(lens, dtype=torch.int32, device="cuda"), table, window=W, sinks=sinks)
    assert sdp.poll_status() == sdp.SDP_OK
    for s in range(2):
        r = slice(int(cu[s]), int(cu[s + 1]))
        ro, _, mag, dot = reference(last[s][:, None], kg[r].transpose(0, 1), vg[r].transpose(0, 1), W, sinks, 1 / math.sqrt(D))
        e = 2.0 ** -8 * dot / math.sqrt(D)
        assert ((o[s][:, None].double() - ro).abs() <= 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2 * e) * mag * 1.01).all()
