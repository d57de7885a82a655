"""The forms of the sliding-window kernels that larger batches run (several units a CTA, one CTA or a pair of them a
unit), every row against the definition in 64 bits: units of many tiles, maxima that move late in a unit, masks of wide
windows, first tokens over several tiles, ragged packed batches. Tolerances as in test_window.
"""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp
from test_window import DTYPES, check

# heads, head dim, debug flags: one CTA a unit at D = 128; pairs of CTAs; one CTA a unit for odd groups, and by the flag
FORMS = {"many_d128": (16, 4, 128, 0), "many_d128_odd": (15, 5, 128, 0), "pairs_d256": (16, 4, 256, 0),
         "pairs_d256_two": (16, 8, 256, 0), "many_d256_odd": (15, 5, 256, 0), "many_d256": (16, 4, 256, 2)}


def growing(k, lens):
    """Keys that get louder along each sequence, so that a row's maximum moves up to its last tiles."""
    ramp = torch.cat([0.4 + 2.2 * torch.arange(n, device=k.device) / max(n, 1) for n in lens])
    return (k * ramp[:, None, None]).to(k.dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("Sq,Skv,window,sinks", [(2500, 2500, 800, 129), (2500, 2500, 9000, 3), (1700, 4100, 1300, 0),
                                                (2300, 900, 257, 500), (2560, 2560, 128, 128), (1300, 6000, 6000, 0)])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_dense(form, Sq, Skv, window, sinks, dt):
    Hq, Hkv, D, flags = FORMS[form]
    assert -(-Sq // 128) * Hq > 152  # more units than SMs
    dtype = DTYPES[dt]
    g = torch.Generator(device="cuda").manual_seed(Sq + Skv + window)
    q = torch.randn(1, Hq, Sq, D, device="cuda", generator=g).to(dtype)
    k, v = (torch.randn(1, Hkv, Skv, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    k = growing(k[0].transpose(0, 1), [Skv]).transpose(0, 1)[None].contiguous()
    old = sdp.set_debug_flags(flags)
    try:
        o, lse = sdp.fwd_window(q, k, v, window, sinks=sinks)
        assert sdp.poll_status() == sdp.SDP_OK
    finally:
        sdp.set_debug_flags(old)
    G = Hq // Hkv
    for n in range(Hkv):
        h = slice(n * G, (n + 1) * G)
        check(o[0, h], lse[0, h], q[0, h], k[0, n:n + 1], v[0, n:n + 1], window, sinks, 1 / math.sqrt(D), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("window,sinks,dt", [(300, 5, "bf16"), (100000, 0, "fp16"), (129, 200, "fp16")])
def test_ragged_packed_batches(form, window, sinks, dt):
    """Over 32 sequences, empty and keyless ones among them, rows before the first key, chunks behind prefixes."""
    Hq, Hkv, D, flags = FORMS[form]
    dtype = DTYPES[dt]
    c = torch.Generator().manual_seed(window + D)
    lq = torch.randint(0, 500, (75,), generator=c)
    lk = (lq + torch.randint(-200, 700, (75,), generator=c)).clamp_min(0)
    lq[[0, 33, 34, 74]] = 0
    lk[[7, 40]] = 0
    lq[50], lk[50] = 1500, 3500
    g = torch.Generator(device="cuda").manual_seed(window)
    q = torch.randn(int(lq.sum()), Hq, D, device="cuda", generator=g).to(dtype)
    k, v = (torch.randn(int(lk.sum()), Hkv, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    k = growing(k, lk.tolist())
    cq, ck = (torch.cat((torch.zeros(1, dtype=torch.int64), x.cumsum(0))).int().cuda() for x in (lq, lk))
    o, lse = torch.full_like(q, math.nan), torch.full((Hq, len(q)), math.nan, device="cuda")
    old = sdp.set_debug_flags(flags)
    try:
        sdp.fwd_varlen_window(q, k, v, cq, ck, 1500, window, sinks=sinks, out=o, lse=lse)
        assert sdp.poll_status() == sdp.SDP_OK
    finally:
        sdp.set_debug_flags(old)
    a = b = 0
    for n, m in zip(lq.tolist(), lk.tolist()):
        if n:
            check(o[a:a + n].transpose(0, 1), lse[:, a:a + n], q[a:a + n].transpose(0, 1), k[b:b + m].transpose(0, 1),
                  v[b:b + m].transpose(0, 1), window, sinks, 1 / math.sqrt(D), dtype)
        a, b = a + n, b + m


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 128), (2, 1, 256), (160, 40, 128), (160, 40, 256), (159, 53, 256)],
                         ids=["one_d128", "one_d256", "many_d128", "pairs_d256", "many_d256"])
@pytest.mark.parametrize("flags", [0, 32], ids=["compact", "full_grid"])
@pytest.mark.parametrize("cq,ck,max_q,bad", [
    ((0, 100, 301), (0, 100, 300), 200, 1), ((0, 100, 300), (0, 200, 100), 200, 1), ((-1, 100, 300), (0, 100, 300), 200, 0),
    ((0, 20, 300), (0, 100, 300), 100, 1), ((0, 100, 300), (0, 100, 301), 200, 1), ((0, 100, 300), (-5, 100, 300), 200, 0)])
def test_a_bad_sequence_is_left_alone_and_the_other_is_right(Hq, Hkv, D, flags, cq, ck, max_q, bad):
    g = torch.Generator(device="cuda").manual_seed(D)
    q = torch.randn(300, Hq, D, device="cuda", generator=g).half()
    k, v = (torch.randn(300, Hkv, D, device="cuda", generator=g).half() for _ in range(2))
    o, lse = torch.full_like(q, 5), torch.full((Hq, 300), 5.0, device="cuda")
    tq, tk = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cq, ck))
    old = sdp.set_debug_flags(flags)
    try:
        sdp.fwd_varlen_window(q, k, v, tq, tk, max_q, 64, sinks=2, out=o, lse=lse)
        assert sdp.poll_status() == sdp.SDP_ERR_BAD_SEQLENS
    finally:
        sdp.set_debug_flags(old)
    rows = slice(max(cq[bad], 0), min(cq[bad + 1], 300))
    assert (o[rows] == 5).all() and (lse[:, rows] == 5).all()
    s = 1 - bad
    r, t = slice(cq[s], cq[s + 1]), slice(ck[s], ck[s + 1])
    check(o[r].transpose(0, 1), lse[:, r], q[r].transpose(0, 1), k[t].transpose(0, 1), v[t].transpose(0, 1), 64, 2,
          1 / math.sqrt(D), torch.float16)
