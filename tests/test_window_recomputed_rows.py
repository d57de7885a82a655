"""Rows that a value which is not finite makes the sliding-window kernels compute again: such a row takes far longer
than a tile, and the launch has to end within the limit of its waits all the same, with every row right.

Tolerances as in test_window.
"""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp
from test_window import DTYPES, reference


@pytest.mark.gpu
@pytest.mark.parametrize("D,Hq,Hkv,dt", [(128, 8, 2, "bf16"), (256, 8, 2, "fp16"), (256, 9, 3, "bf16")],
                         ids=["many_d128", "pairs_d256", "many_d256"])
@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
def test_many_recomputed_rows_over_a_long_window(D, Hq, Hkv, dt, packed):
    """Every unit of several a CTA has all its rows computed again: 128 rows of some 4000 keys, milliseconds a unit,
    with 4 ms for a wait. A value's one channel is infinite, so that the others' results are known."""
    dtype, S, W, sinks = DTYPES[dt], 9000, 4000, 3
    g = torch.Generator(device="cuda").manual_seed(D + Hq)
    q = torch.randn(1, Hq, S, D, device="cuda", generator=g).to(dtype)
    k, v = (torch.randn(1, Hkv, S, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    clean = v.clone()
    v[:, :, 1::512, 5] = math.inf
    if packed:
        cu = torch.tensor([0, S], dtype=torch.int32, device="cuda")
        args = [x[0].transpose(0, 1).contiguous() for x in (q, k, v)] + [cu, cu, S]
        call = sdp.fwd_varlen_window
    else:
        args, call = [q, k, v], sdp.fwd_window
    call(*args, W, sinks=sinks)
    torch.cuda.synchronize()
    old = sdp.set_wait_timeout_ms(4)
    try:
        o, lse = call(*args, W, sinks=sinks)
        assert sdp.poll_status() == sdp.SDP_OK
    finally:
        sdp.set_wait_timeout_ms(old)
    o = o.transpose(0, 1) if packed else o[0]
    lse = lse if packed else lse[0]
    eps, scale = torch.finfo(dtype).eps, 1 / math.sqrt(D)
    rest = [c for c in range(D) if c != 5]
    for h in (0, Hq - 1):
        n = h // (Hq // Hkv)
        ro, rl, mag, dot = reference(q[0, h:h + 1], k[0, n:n + 1], clean[0, n:n + 1], W, sinks, scale)
        e = 2.0 ** -20 * scale * dot
        tol = eps / 2 * ro.abs() + (eps / 2 + 2.0 ** -19) * mag + 2 * e * float(clean.double().abs().max()) + 2.0 ** -24
        bad = ((o[h:h + 1].double() - ro).abs() > tol) | torch.isnan(o[h:h + 1])
        assert not bad[..., rest].any(), (int(bad[..., rest].sum()), bad[..., rest].nonzero()[:4].tolist())
        assert (o[h, 1:, 5] == math.inf).all()  # each row from the second on sees one
        assert ((lse[h].double() - rl[0]).abs() <= e + 2.0 ** -19 * (1 + rl[0].abs())).all()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
def test_recomputed_rows_of_ragged_units(D):
    """Marked rows in some units of a packed batch with empty and keyless sequences, found again from the offsets:
    values that are not finite in sight of some rows only, and the first of the next sequence's keys in a tile."""
    g = torch.Generator().manual_seed(D)
    lq = torch.randint(0, 400, (60,), generator=g)
    lk = lq + torch.randint(-100, 300, (60,), generator=g)
    lq[[3, 40]], lk[[7, 41]] = 0, 0
    lk = lk.clamp_min(0)
    Hq, Hkv, W, sinks, dtype = 6, 2, 90, 2, torch.float16
    q = torch.randn(int(lq.sum()), Hq, D, generator=g).to(dtype).cuda()
    k, v = (torch.randn(int(lk.sum()), Hkv, D, generator=g).to(dtype).cuda() for _ in range(2))
    hit = torch.randint(0, int(lk.sum()), (25,), generator=g).cuda()
    v[hit, 1, 9] = math.nan
    cq, ck = (torch.cat((torch.zeros(1, dtype=torch.int64), x.cumsum(0))).int().cuda() for x in (lq, lk))
    o, lse = sdp.fwd_varlen_window(q, k, v, cq, ck, 400, W, sinks=sinks)
    assert sdp.poll_status() == sdp.SDP_OK
    rest = [c for c in range(D) if c != 9]
    eps, scale = torch.finfo(dtype).eps, 1 / math.sqrt(D)
    a = b = 0
    for n, m in zip(lq.tolist(), lk.tolist()):
        if n:
            vs = v[b:b + m].transpose(0, 1)
            nan = torch.isnan(vs[:, :, 9])
            ro, rl, mag, dot = reference(q[a:a + n].transpose(0, 1), k[b:b + m].transpose(0, 1), vs.nan_to_num(0), W, sinks, scale)
            x = o[a:a + n].transpose(0, 1)
            vmax = float(vs.nan_to_num(0).double().abs().max()) if m else 0.0
            tol = eps / 2 * ro.abs() + (eps / 2 + 2.0 ** -19) * mag + 2.0 ** -19 * scale * dot * vmax + 2.0 ** -24
            off = ((x.double() - ro).abs() > tol) | torch.isnan(x)
            assert not off[..., rest].any()
            p = torch.arange(m - n, m, device="cuda")[:, None]
            j = torch.arange(m, device="cuda")[None]
            seen = (j <= p) & ((j > p - W) | (j < sinks))
            want = (seen[None] & nan[:, None].repeat_interleave(Hq // Hkv, 0)).any(-1)
            assert torch.equal(torch.isnan(x[..., 9]), want)
            assert not off[..., 9][~want].any()
        a, b = a + n, b + m
