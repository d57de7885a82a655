"""sdp_qk_norm_rope: refusals (CPU), and every element against the definition in 64 bits (GPU).

Tolerance of an element y = a c - b s (or its partner): half a step of the stored type,
finfo.eps / 2 * |y| (2^-25 absolute where fp16 is subnormal), plus the fp32 arithmetic before it,
at most 2e-6 * mscale * (|a| + |b|): the sum of squares (8 + log2 terms in sequence, 2^-21), rsqrt
(2 ulp, 2^-22), two products (2^-23), the angle from its 32-bit fraction in fp32 (pi * 2^-25),
sincospif (2 ulp) and the products of the rotation (2^-23) add to less than 14 * 2^-23.
"""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the frequencies and the refusals (CPU)


def test_frequencies():
    f = sdp.rope_inv_freq(128, 10000.0)
    assert f.dtype == torch.float64 and f.shape == (64,)
    assert f[0] == 1 and abs(f[63].item() - 10000.0 ** (-126 / 128)) < 1e-18
    lin = sdp.rope_inv_freq(128, 10000.0, scaling="linear", factor=4)
    assert torch.equal(lin, f / 4)
    ntk = sdp.rope_inv_freq(128, 10000.0, scaling="ntk", factor=4)
    assert ntk[0] == 1 and abs(ntk[63] / f[63] - 0.25) < 1e-12
    yarn = sdp.rope_inv_freq(128, 10000.0, scaling="yarn", factor=4, original_length=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(yarn[turns > 64], f[turns > 64])
    assert torch.allclose(yarn[turns < 0.9], f[turns < 0.9] / 4, rtol=1e-12, atol=0)
    assert (yarn[1:] < yarn[:-1]).all()
    assert sdp.rope_inv_freq(0).numel() == 0
    for bad in (dict(dim=7), dict(dim=8, scaling="other"), dict(dim=8, factor=0.5),
                dict(dim=8, scaling="yarn", factor=2.0)):
        with pytest.raises(ValueError):
            sdp.rope_inv_freq(**bad)


def test_table_holds_the_fraction_of_a_turn():
    f = sdp.rope_inv_freq(64, 5e6)
    t = sdp.rope_table(f, mscale=1.5)
    assert t.mscale == 1.5 and t.turns.dtype == torch.int64
    for i in (0, 1, 17, 31):
        want = f[i].item() / (2 * math.pi)
        got = (t.turns[i].item() % 2 ** 64) / 2.0 ** 64
        assert abs(got - want) <= 2.0 ** -52 * want + 2.0 ** -64  # the last place of the fraction
    big = sdp.rope_table(torch.tensor([100.0, -1.0], dtype=torch.float64))  # more than a turn; backwards
    for i, x in enumerate((100.0, -1.0)):
        assert abs((big.turns[i].item() % 2 ** 64) / 2.0 ** 64 - (x / (2 * math.pi)) % 1) < 1e-14
    with pytest.raises(ValueError):
        sdp.rope_table(torch.zeros(2, 2))
    with pytest.raises(ValueError):
        sdp.rope_table(torch.zeros(2, dtype=torch.int64))


A = 0x10000  # stand-in addresses: validation returns before anything is read


def c_call(**kw):
    from gqa_flash_attention_gb300 import serving
    a = dict(q=A, qs=(0, 512, 128), k=2 * A, ks=(0, 512, 128), qo=3 * A, qos=(0, 512, 128), ko=4 * A,
             kos=(0, 512, 128), pos=5 * A, ps=(0, 1), p64=0, turns=6 * A, R=128, mscale=1.0, wq=0, wk=0, w32=0,
             eps=1e-6, il=0, B=1, S=4, Hq=4, Hkv=2, D=128, dtype=0)
    a.update(kw)
    return serving._lib().sdp_qk_norm_rope(
        a["q"], *a["qs"], a["k"], *a["ks"], a["qo"], *a["qos"], a["ko"], *a["kos"], a["pos"], *a["ps"], a["p64"],
        a["turns"], a["R"], a["mscale"], a["wq"], a["wk"], a["w32"], a["eps"], a["il"], a["B"], a["S"], a["Hq"],
        a["Hkv"], a["D"], a["dtype"], 0)


@pytest.mark.parametrize("kw,code", [
    (dict(D=64), sdp.SDP_ERR_UNSUPPORTED),
    (dict(dtype=2), sdp.SDP_ERR_UNSUPPORTED),
    (dict(R=24), sdp.SDP_ERR_INVALID_ARG),
    (dict(R=144), sdp.SDP_ERR_INVALID_ARG),
    (dict(R=-16), sdp.SDP_ERR_INVALID_ARG),
    (dict(B=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(q=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(ko=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(pos=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(turns=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(eps=math.nan), sdp.SDP_ERR_INVALID_ARG),
    (dict(eps=-1.0), sdp.SDP_ERR_INVALID_ARG),
    (dict(mscale=math.inf), sdp.SDP_ERR_INVALID_ARG),
    (dict(q=A + 8), sdp.SDP_ERR_ALIGNMENT),
    (dict(ks=(0, 512, 124)), sdp.SDP_ERR_ALIGNMENT),
    (dict(wq=A + 4), sdp.SDP_ERR_ALIGNMENT),
    (dict(pos=A + 4, p64=1), sdp.SDP_ERR_ALIGNMENT),
    (dict(B=1 << 16, S=1 << 16), sdp.SDP_ERR_OVERFLOW),
    (dict(S=0), sdp.SDP_OK),
    (dict(B=0, q=0), sdp.SDP_OK),
])
def test_c_call_refuses_before_any_launch(kw, code):
    from gqa_flash_attention_gb300 import build
    build.build()
    assert c_call(**kw) == code


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 2, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        sdp.qk_norm_rope(x, x, None, None)
    with pytest.raises(ValueError):
        sdp.qk_norm_rope(x[0], None, None, None)


# ------------------------------------------------------------------ against the definition (GPU)


def reference(x, w, eps, pos, inv_freq, mscale, interleaved):
    """x [..., H, D] with pos [...], in 64 bits: values, and |a| + |b| of each element's pair."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    size = y.abs()
    R = 0 if inv_freq is None else 2 * len(inv_freq)
    if R:
        # the angle modulo a turn with whole numbers: fp64 products lose it too at the farthest positions
        t = (pos.double()[..., None, None] * inv_freq)
        if pos.abs().max() > 1 << 22:
            num = (inv_freq / (2 * math.pi)).tolist()
            from fractions import Fraction
            fr = [Fraction(v) for v in num]
            t = torch.tensor([[float((int(p) * f) % 1) for f in fr] for p in pos.flatten().tolist()],
                             dtype=torch.float64).view(*pos.shape, 1, -1) * (2 * math.pi)
        c, s = torch.cos(t) * mscale, torch.sin(t) * mscale
        ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
        ib = ia + 1 if interleaved else ia + R // 2
        a, b = y[..., ia].clone(), y[..., ib].clone()
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        size = size.clone()
        size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * abs(mscale)
    return y, size


def check(got, want, size, dtype):
    got = got.double().cpu()
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -25 + 2e-6 * size
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), (got - want).abs()[bad].max())


CASES = []
for dt in ("fp16", "bf16"):
    CASES += [
        # T, Hq, Hkv, D, R, norm, interleaved, pos64, w32
        (1, 4, 1, 128, 128, True, False, False, False, dt),
        (7, 32, 8, 128, 128, True, True, False, True, dt),
        (3, 5, 3, 128, 64, False, False, True, False, dt),
        (130, 3, 3, 128, 16, True, True, True, False, dt),
        (2, 32, 2, 256, 256, True, False, False, True, dt),
        (33, 7, 1, 256, 64, False, True, False, False, dt),
        (65, 1, 1, 256, 96, True, False, True, False, dt),
        (5, 2, 2, 128, 0, True, False, False, False, dt),
        (700, 32, 8, 128, 96, True, False, False, False, dt),
        (301, 40, 8, 256, 128, True, True, False, False, dt),
    ]


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hkv,D,R,norm,interleaved,pos64,w32,dt", CASES)
def test_packed_rows(T, Hq, Hkv, D, R, norm, interleaved, pos64, w32, dt):
    g = torch.Generator().manual_seed(T * 131 + D + R)
    dtype = DTYPES[dt]
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).to(dtype)  # a fused projection's rows
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int64 if pos64 else torch.int32)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(torch.float32 if w32 else dtype) for _ in range(2)]
    f = sdp.rope_inv_freq(R, 10000.0) if R else None
    dev = qkv.cuda()
    q, k = dev[:, :Hq * D].view(T, Hq, D), dev[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    before = dev.clone()
    table = sdp.rope_table(f.cuda(), mscale=1.25) if R else None
    qo, ko = sdp.qk_norm_rope(q, k, pos.cuda() if R else None, table, w[0].cuda() if norm else None,
                              w[1].cuda() if norm else None, eps=1e-5, interleaved=interleaved)
    assert qo.is_contiguous() and ko.is_contiguous()
    for got, x, wi in ((qo, q, w[0]), (ko, k, w[1])):
        want, size = reference(x.cpu(), wi if norm else None, 1e-5, pos, f, 1.25, interleaved)
        check(got, want, size, dtype)
    assert torch.equal(dev, before)
    # in place, and with only one of the two normed
    qo2, ko2 = sdp.qk_norm_rope(q, k, pos.cuda() if R else None, table, w[0].cuda() if norm else None,
                                w[1].cuda() if norm else None, eps=1e-5, interleaved=interleaved, q_out=q, k_out=k)
    assert qo2 is q and torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(dev[:, (Hq + Hkv) * D:], before[:, (Hq + Hkv) * D:])  # V's columns


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("interleaved", [True, False])
def test_dense_batches(shared, interleaved):
    g = torch.Generator().manual_seed(9)
    B, S, Hq, Hkv, D = 3, 37, 6, 2, 128
    x = torch.randn(B, S, Hq + Hkv, D, generator=g).to(torch.bfloat16)
    pos = torch.arange(S) if shared else torch.randint(0, 5000, (B, S), generator=g)
    f = sdp.rope_inv_freq(D, 10000.0)
    dev = x.cuda()
    q, k = dev[:, :, :Hq].transpose(1, 2), dev[:, :, Hq:].transpose(1, 2)  # [B, H, S, D] views
    qo, ko = sdp.qk_norm_rope(q, k, pos.cuda(), sdp.rope_table(f.cuda()), interleaved=interleaved)
    assert qo.shape == (B, Hq, S, D) and qo.is_contiguous()
    p = pos.expand(B, S)
    for got, h in ((qo, slice(0, Hq)), (ko, slice(Hq, None))):
        want, size = reference(x[:, :, h], None, 0, p, f, 1.0, interleaved)
        check(got, want.transpose(1, 2), size.transpose(1, 2), torch.bfloat16)


@pytest.mark.gpu
def test_far_and_negative_positions():
    pos = torch.tensor([0, 1, -1, 1 << 24, (1 << 31) - 1, -(1 << 31), 12345678, -777])
    f = sdp.rope_inv_freq(128, 10000.0)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(len(pos), 2, 128, generator=g).to(torch.float16)
    for p in (pos.int(), pos, pos * (1 << 20)):
        qo, none = sdp.qk_norm_rope(x.cuda(), None, p.cuda(), sdp.rope_table(f.cuda()))
        assert none is None
        want, size = reference(x, None, 0, p, f, 1.0, False)
        # f itself is rounded to 2^-53 of a turn's fraction, so position 2^51 has lost its angle:
        # 2 pi * |p| * 2^-53 more
        more = 2 * math.pi * p.abs().double()[:, None, None] * 2.0 ** -53
        got = qo.double().cpu()
        tol = torch.finfo(torch.float16).eps / 2 * want.abs() + 2.0 ** -25 + (2e-6 + more) * size
        assert ((got - want).abs() <= tol).all()


@pytest.mark.gpu
def test_one_weight_only_and_zero_rows():
    g = torch.Generator().manual_seed(4)
    q, k = torch.randn(9, 3, 128, generator=g).half(), torch.randn(9, 3, 128, generator=g).half()
    q[4] = 0  # a zero row: eps keeps it 0
    w = (1 + torch.randn(128, generator=g)).half()
    qo, ko = sdp.qk_norm_rope(q.cuda(), k.cuda(), None, None, q_weight=w.cuda())
    want, size = reference(q, w, 1e-6, None, None, 1.0, False)
    check(qo, want, size, torch.float16)
    assert (qo[4] == 0).all() and torch.equal(ko.cpu(), k)
    qo, ko = sdp.qk_norm_rope(q.cuda(), k.cuda(), None, None, k_weight=w.cuda())
    want, size = reference(k, w, 1e-6, None, None, 1.0, False)
    check(ko, want, size, torch.float16)
    assert torch.equal(qo.cpu(), q)
    e = torch.empty(0, 3, 128, device="cuda", dtype=torch.float16)
    assert sdp.qk_norm_rope(e, None, None, None)[0].shape == (0, 3, 128)


@pytest.mark.gpu
def test_streams_graphs_and_refusals():
    x = torch.randn(64, 8, 128, device="cuda").to(torch.bfloat16)
    f = sdp.rope_inv_freq(64, device="cuda")
    t = sdp.rope_table(f)
    pos = torch.arange(64, device="cuda")
    want, _ = sdp.qk_norm_rope(x, None, pos, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = sdp.qk_norm_rope(x, None, pos, t, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sdp.qk_norm_rope(x, None, pos, t, q_out=out)
    for shift in (0, 5):
        pos.copy_(torch.arange(64, device="cuda") + shift)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sdp.qk_norm_rope(x, None, pos, t)[0])
    bad = [
        dict(q=x.float()), dict(q=x[..., :64]), dict(q=x.transpose(1, 2)), dict(q=x, k=x.half()), dict(q=x, k=x[:5]),
        dict(q=x, positions=pos[:3]), dict(q=x, positions=pos.float()), dict(q=x, positions=pos.cpu()),
        dict(q=x, table=sdp.rope_table(f.cpu())), dict(q=x, q_weight=torch.ones(64, device="cuda")),
        dict(q=x, k_weight=torch.ones(128, device="cuda")), dict(q=x, q_out=x[:5]),
        dict(q=x, q_weight=torch.ones(128, device="cuda", dtype=torch.float16)),
    ]
    for kw in bad:
        a = dict(k=None, positions=pos, table=t)
        a.update(kw)
        with pytest.raises((ValueError, sdp.SdpError)):
            sdp.qk_norm_rope(**a)
    y = x.clone().requires_grad_()
    with pytest.raises(ValueError):
        sdp.qk_norm_rope(y, None, pos, t)
    with torch.no_grad():
        sdp.qk_norm_rope(y, None, pos, t)
