"""qk_norm_rope on rows whose squares leave fp32's range, in bf16: every element against the definition in 64 bits.
Tolerance as in test_qk_norm_rope, with bf16's smallest normal number for results below it.
"""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp
from test_qk_norm_rope import reference


def check(got, want, size):
    got = got.double().cpu()
    tol = 2.0 ** -8 * want.abs() + 2e-6 * size + 2.0 ** -126
    bad = ((got - want).abs() > tol) | torch.isnan(got)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [1e-6, 0.0, 1e-30, 1e4])
@pytest.mark.parametrize("D,R,interleaved,w32", [(128, 128, False, False), (128, 64, True, True), (256, 96, False, True),
                                                (256, 256, True, False), (128, 0, False, False)])
def test_rows_of_every_size(D, R, interleaved, w32, eps):
    """Rows of 2^-120 to 2^126, ordinary ones between them; heads that do not fill a warp's pass."""
    g = torch.Generator().manual_seed(D + R)
    e = torch.tensor([-120, 0, -70, 126, 1, 64, 20, 90, -45, 62, 100, -3, 124])
    x = torch.randn(len(e), 5, D, generator=g).clamp(-1.9, 1.9)
    x = (x.double() * 2.0 ** e.double()[:, None, None]).bfloat16()
    x[3, 1] = 0
    x[3, 1, 7] = torch.finfo(torch.bfloat16).max
    if eps == 0:
        x[x == 0] = 2.0 ** -100
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(torch.float32 if w32 else torch.bfloat16) for _ in range(2)]
    pos = torch.randint(0, 1 << 20, (len(e),), generator=g)
    f = sdp.rope_inv_freq(R, 10000.0) if R else None
    table = sdp.rope_table(f.cuda(), mscale=1.25) if R else None
    q, k = x[:, :4], x[:, 4:]
    dev = x.cuda()
    qo, ko = sdp.qk_norm_rope(dev[:, :4], dev[:, 4:], pos.cuda() if R else None, table, w[0].cuda(), w[1].cuda(), eps=eps,
                              interleaved=interleaved)
    for got, y, wi in ((qo, q, w[0]), (ko, k, w[1])):
        check(got, *reference(y, wi, eps, pos, f, 1.25, interleaved))


@pytest.mark.gpu
def test_a_rows_bits_do_not_depend_on_its_neighbours():
    """D = 128: two rows a pass of a warp, one of them out of range; infinities and NaN stay in their own row."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 8, 128, generator=g).bfloat16().cuda()
    w = (1 + torch.randn(128, generator=g)).bfloat16().cuda()
    pos, table = torch.arange(40).cuda(), sdp.rope_table(sdp.rope_inv_freq(128).cuda())
    want, _ = sdp.qk_norm_rope(x, None, pos, table, w)
    y = x.clone()
    y[:, 1::2] *= 1e30
    y[7, 3, 5], y[8, 5, 6] = math.inf, math.nan
    got, _ = sdp.qk_norm_rope(y, None, pos, table, w)
    assert torch.equal(got[:, 0::2], want[:, 0::2])
    assert torch.isnan(got[8, 5]).all()
    assert torch.isnan(got[7, 3, [5, 69]]).all()  # inf / inf, in the pair that holds it; the others over infinity
    assert (got[7, 3, [c for c in range(128) if c % 64 != 5]] == 0).all()
    got[7, 3], got[8, 5] = 0, 0
    assert torch.isfinite(got).all()
    # rows in range as before: a power of two changes no bit of a row normed without an eps
    a, _ = sdp.qk_norm_rope(x, None, pos, table, w, eps=0.0)
    b, _ = sdp.qk_norm_rope(x * 2.0 ** 80, None, pos, table, w, eps=0.0)
    c, _ = sdp.qk_norm_rope(x * 2.0 ** -80, None, pos, table, w, eps=0.0)
    assert ((a.double() - b.double()).abs() <= 2.0 ** -7 * a.double().abs()).all()
    assert torch.equal(b, c)
