"""Attention over the 16-bit paged cache with shared prefixes (sdp_fwd_cache16): refusals on the CPU; on the GPU every row
against the definition in 64 bits.

Tolerance, for a row with scores s_j, weights w_j (of sum 1) and values v: a score's products are exact in fp32, their sum
is accumulated by the tensor core (each of D / 16 steps may drop a bit of the running sum's last place): with its scaling and
the exponential, each weight is off by a factor 1 + 2 e at most, e = |scale| max_j sum_c |q_c k_jc| * 2^-18
+ 2^-21 * (1 + max |s|). A weight is rounded to dtype for the product with V (half a step, finfo.eps / 2 of it; fp16: among
the subnormals 2^-25 of weights whose sum is 1 or more before they are divided), the sum of l is not. O's steps, n / 16 and
the parts' joining, each drop 2^-23. So with W = sum_j w_j |v_j|:
    finfo.eps / 2 * |o|  +  (finfo.eps / 2 + 4 e + (n / 16 + 64) 2^-23) * W * (1 + 2^-6)
    + (fp16) n 2^-25 max |v| + 2^-25;
the log-sum-exp by 2 e + 2^-20 (1 + |lse|).
"""
import math

import pytest
import torch

import gqa_flash_attention_gb300 as sdp

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
A = 0x10000


def c_call(**kw):
    from gqa_flash_attention_gb300 import serving
    a = dict(q=A, kc=2 * A, vc=3 * A, P=8, page=16, table=4 * A, ts=4, mp=4, lens=5 * A, ptable=6 * A, ps=4, pp=4,
             plens=7 * A, cu=8 * A, ng=2, o=9 * A, lse=10 * A, nseq=2, rows=1, Hq=8, Hkv=2, D=128, scale=0.1, dtype=0,
             ws=11 * A, wb=1 << 30)
    a.update(kw)
    return serving._lib().sdp_fwd_cache16(*a.values(), 0)


@pytest.mark.parametrize("kw,code", [
    (dict(D=192), sdp.SDP_ERR_UNSUPPORTED),
    (dict(dtype=2), sdp.SDP_ERR_UNSUPPORTED),
    (dict(rows=33), sdp.SDP_ERR_UNSUPPORTED),
    (dict(rows=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(nseq=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(Hq=7), sdp.SDP_ERR_INVALID_ARG),
    (dict(ng=-1), sdp.SDP_ERR_INVALID_ARG),
    (dict(page=8), sdp.SDP_ERR_INVALID_ARG),
    (dict(P=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(mp=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(pp=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(ptable=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(plens=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(cu=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(scale=math.nan), sdp.SDP_ERR_INVALID_ARG),
    (dict(q=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(vc=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(ws=0), sdp.SDP_ERR_INVALID_ARG),
    (dict(o=A), sdp.SDP_ERR_INVALID_ARG),
    (dict(o=3 * A), sdp.SDP_ERR_INVALID_ARG),
    (dict(kc=2 * A + 8), sdp.SDP_ERR_ALIGNMENT),
    (dict(lse=10 * A + 2), sdp.SDP_ERR_ALIGNMENT),
    (dict(plens=7 * A + 2), sdp.SDP_ERR_ALIGNMENT),
    (dict(ws=11 * A + 4), sdp.SDP_ERR_ALIGNMENT),
    (dict(mp=1 << 27), sdp.SDP_ERR_OVERFLOW),
    (dict(pp=1 << 27), sdp.SDP_ERR_OVERFLOW),
    (dict(P=1 << 30, Hkv=8), sdp.SDP_ERR_OVERFLOW),
    (dict(nseq=1 << 29), sdp.SDP_ERR_OVERFLOW),
    (dict(nseq=1 << 20, mp=1 << 20, ng=0), sdp.SDP_ERR_OVERFLOW),  # tiles of all problems
])
def test_c_call_refuses_before_any_launch(kw, code):
    from gqa_flash_attention_gb300 import build, serving
    build.build()
    assert c_call(**kw) == code
    if set(kw) <= {"D", "dtype", "rows", "nseq", "Hq", "ng"}:
        a = dict(nseq=2, rows=1, Hq=8, Hkv=2, D=128, dtype=0, ng=2)
        a.update(kw)
        assert serving._lib().sdp_fwd_cache16_workspace_bytes(*a.values()) == code


def test_workspace_type():
    for dtype in (torch.float32, None):
        with pytest.raises(ValueError):
            sdp.cache16_workspace_bytes(1, 1, 8, 2, 128, dtype)


# ------------------------------------------------------------------ GPU


class Batch:
    """Sequences of lengths `lens` (with their prefixes), groups by offsets `cu` with prefixes of lengths `prefix`, in a pool
    whose other places hold NaN and infinities; a prefix's part of a sequence's own page is not written."""

    def __init__(self, lens, cu, prefix, rows, Hq, Hkv, D, page, dtype, seed=0, kscale=1.0, own_pages=()):
        g = torch.Generator().manual_seed(seed + 7 * sum(lens) + D)
        self.lens, self.cu, self.prefix, self.rows, self.dtype = lens, cu, prefix, rows, dtype
        self.group = [-1] * len(lens)
        for k in range(len(prefix)):
            for s in range(cu[k], cu[k + 1]):
                self.group[s] = k

        def rows_of(n):
            k = kscale * torch.randn(n, Hkv, D, generator=g)
            k[:, :, 5] += 2
            v = torch.randn(n, Hkv, D, generator=g) * torch.exp(torch.randn(n, 1, 1, generator=g)) + 0.3
            return k.to(dtype), v.to(dtype)

        shared = [rows_of(p) for p in prefix]
        need = [-(-n // page) for n in lens]
        first = [-(-p // page) for p in prefix]
        pool = sum(need) + sum(first) + 2
        order = torch.randperm(pool, generator=g).int()
        self.k = torch.full((pool, Hkv, page, D), math.nan, dtype=dtype)
        self.v = torch.full((pool, Hkv, page, D), math.nan, dtype=dtype)
        self.v[:, :, 1::2] = math.inf
        self.table = torch.full((len(lens), max(1, max(need))), -7, dtype=torch.int32)
        self.prefix_table = torch.full((max(1, len(prefix)), max([1, *first])), -9, dtype=torch.int32)
        at = 0
        for k, n in enumerate(first):
            self.prefix_table[k, :n] = order[at:at + n]
            at += n
            t = torch.arange(prefix[k])
            ids = self.prefix_table[k, t // page].long()
            self.k[ids, :, t % page], self.v[ids, :, t % page] = shared[k]
        self.rows_kv = []
        for s, n in enumerate(lens):
            k = self.group[s]
            P = prefix[k] if k >= 0 else 0
            alone = k < 0 or n < P + rows - 1 or cu[k + 1] - cu[k] == 1 or P == 0 or s in own_pages
            if alone:
                P = min(P, n)
            kk, vv = rows_of(max(0, n - P))
            if P:
                kk, vv = torch.cat((shared[k][0][:P], kk)), torch.cat((shared[k][1][:P], vv))
            self.rows_kv.append((kk, vv))
            lo = 0 if alone else P  # what the call may read of the sequence's own pages
            if n > lo:
                pages = slice(lo // page, need[s])
                count = need[s] - lo // page
                self.table[s, pages] = order[at:at + count]
                at += count
                t = torch.arange(lo, n)
                ids = self.table[s, t // page].long()
                self.k[ids, :, t % page], self.v[ids, :, t % page] = kk[lo:], vv[lo:]
        self.q = torch.randn(len(lens), rows, Hq, D, generator=g).to(dtype)

    def args(self, device="cuda"):
        a = dict(q=self.q.to(device), cache=sdp.Cache16(self.k.to(device), self.v.to(device)),
                 cache_lens=torch.tensor(self.lens, dtype=torch.int32, device=device), block_table=self.table.to(device))
        if self.prefix:
            a["prefix_table"] = self.prefix_table.to(device)
            a["prefix_lens"] = torch.tensor(self.prefix, dtype=torch.int32, device=device)
            a["cu_groups"] = torch.tensor(self.cu, dtype=torch.int32, device=device)
        return a

    def check(self, o, lse, scale=None, only=None):
        rows, D = self.rows, self.q.shape[-1]
        scale = 1 / math.sqrt(D) if scale is None else scale
        o, lse = o.double().cpu(), None if lse is None else lse.double().cpu()
        half = torch.finfo(self.dtype).eps / 2
        for s, n in enumerate(self.lens):
            if only is not None and s not in only:
                continue
            k, v = (x.double() for x in self.rows_kv[s])
            G = self.q.shape[2] // k.shape[1]
            q = self.q[s].double()
            kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
            z = torch.einsum("nhd,jhd->nhj", q, kk) * scale
            seen = torch.arange(n)[None] <= torch.arange(n - rows, n)[:, None]
            z = z.masked_fill(~seen[:, None], -math.inf)
            rl = torch.logsumexp(z, -1) if n else torch.full(z.shape[:2], -math.inf, dtype=torch.float64)
            none = rl.isinf()
            assert (o[s][none] == 0).all()
            if lse is not None:
                assert torch.equal(lse[s][none], rl[none])
            if n == 0:
                continue
            w = torch.exp(z - rl.masked_fill(none, 0)[..., None])
            ro, W = torch.einsum("nhj,jhd->nhd", w, vv), torch.einsum("nhj,jhd->nhd", w, vv.abs())
            size = torch.einsum("nhd,jhd->nhj", q.abs(), kk.abs()).amax(-1) * abs(scale)
            top = z.masked_fill(~seen[:, None], 0).abs().amax(-1)
            e = size * 2.0 ** -18 + 2.0 ** -21 * (1 + top)
            tol = (half * ro.abs() + (half + 4 * e[..., None] + (n / 16 + 64) * 2.0 ** -23) * W * (1 + 2.0 ** -6) + 2.0 ** -25
                   + (n * 2.0 ** -25 * vv.abs().amax() if self.dtype == torch.float16 else 0))
            bad = ~((o[s] - ro).abs() <= tol)
            assert not bad.any(), (s, n, int(bad.sum()), bad.nonzero()[:4].tolist(), (o[s] - ro).abs()[bad].max(), tol[bad].max())
            if lse is not None:
                off = (~((lse[s] - rl).abs() <= 2 * e + 2.0 ** -20 * (1 + rl.abs())))[~none]
                assert not off.any(), (s, n, (lse[s] - rl).abs()[~none].max())


CASES = []
for dt in ("fp16", "bf16"):
    CASES += [
        # lens, group offsets, prefix lengths, rows, Hq, Hkv, D, page
        ([1], [0], [], 1, 1, 1, 128, 16, dt),
        ([500], [0], [], 1, 32, 8, 128, 16, dt),
        ([127, 128, 129, 0, 256, 257], [0], [], 1, 8, 2, 128, 64, dt),
        ([77, 0, 0, 1300], [0], [], 1, 16, 1, 256, 64, dt),
        ([700, 40, 2], [0], [], 4, 8, 2, 128, 128, dt),               # rows, one sequence shorter than them
        ([90, 300], [0], [], 32, 14, 2, 256, 16, dt),                 # 224 rows of a KV head: blocks of 18 tokens
        ([100, 400], [0], [], 3, 200, 1, 128, 32, dt),                # a group of more than 128 heads
        ([130, 140, 150], [0, 3], [128], 1, 8, 2, 128, 16, dt),
        ([130, 140, 128], [0, 3], [128], 1, 8, 2, 128, 64, dt),       # one that ends with the prefix
        ([140, 141, 145, 300], [0, 4], [139], 1, 4, 1, 128, 48, dt),  # a prefix that ends inside a page
        ([1100, 1013, 1500], [0, 3], [1007], 2, 7, 1, 256, 128, dt),
        ([600, 590, 0, 100, 700, 601], [0, 6], [590], 3, 8, 8, 128, 32, dt),  # empty and short ones among them
        ([40, 50, 60, 70, 80, 90], [0, 2, 2, 3, 5], [33, 10, 20, 64], 1, 6, 3, 128, 16, dt),  # groups of 2, 0, 1, 2, and one in none
        ([300] * 40, [0, 40], [256], 1, 16, 2, 128, 64, dt),          # 320 rows of a KV head: three blocks
        ([290 + i for i in range(20)], [0, 20], [280], 5, 16, 1, 256, 256, dt),
        ([5000, 5100, 4999], [0, 3], [4990], 1, 32, 2, 256, 64, dt),  # few rows: the prefix cut over many CTAs
        ([3000, 10, 3500, 20], [0], [], 1, 4, 4, 256, 16, dt),
    ]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,cu,prefix,rows,Hq,Hkv,D,page,dt", CASES)
def test_every_row(lens, cu, prefix, rows, Hq, Hkv, D, page, dt):
    b = Batch(lens, cu, prefix, rows, Hq, Hkv, D, page, DTYPES[dt])
    o, lse = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(o, lse)


MORE = [
    # more entries than a CTA has threads: each looks up several
    ([3 + i % 50 for i in range(700)], [0], [], 1, 4, 1, 128, 16, "bf16"),
    ([40 + i % 30 for i in range(1100)], list(range(0, 1101, 2)), [20 + g % 25 for g in range(550)], 2, 2, 1, 256, 16, "fp16"),
    # a block whose last rows have no query, and pages of 80 tokens
    ([1300, 1333, 1290], [0, 3], [1281], 5, 20, 1, 128, 80, "bf16"),
    ([4097, 4200], [0, 2], [4096], 32, 8, 4, 128, 64, "fp16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,cu,prefix,rows,Hq,Hkv,D,page,dt", MORE)
def test_many_entries_and_ragged_blocks(lens, cu, prefix, rows, Hq, Hkv, D, page, dt):
    b = Batch(lens, cu, prefix, rows, Hq, Hkv, D, page, DTYPES[dt])
    o, lse = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("scale,kscale,D", [(0.0, 1.0, 128), (-0.1, 1.0, 256), (0.5, 1.0, 128), (0.02, 16.0, 256), (1e-30, 1.0, 128)])
def test_scales(scale, kscale, D):
    """Scores of 0, of the other sign, and of hundreds, whose maximum moves from tile to tile."""
    b = Batch([700, 900, 650], [0, 3], [600], 2, 8, 2, D, 64, torch.bfloat16, kscale=kscale)
    o, lse = sdp.fwd_cache16(**b.args(), scale=scale)
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(o, lse, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("up", [True, False])
def test_scores_that_grow_or_fall_along_the_keys(D, up):
    """Each tile's maximum above the one before by more than is let pass (or far below it)."""
    b = Batch([2000, 1200], [0, 2], [1000], 1, 4, 1, D, 64, torch.bfloat16)
    for k, v in b.rows_kv:
        n = k.shape[0]
        ramp = torch.arange(n if up else n - 1, -1 if not up else n + n, 1 if up else -1)[:n].double()
        k[:, :, :] = k * 0.25
        k[:, :, 7] = (ramp / 24 - (n / 24 if up else 0)).to(k.dtype)[:, None]
    b.rows_kv[1][0][:1000] = b.rows_kv[0][0][:1000]
    b.rows_kv[1][1][:1000] = b.rows_kv[0][1][:1000]
    b.q[..., 7] = 16.0
    page = b.k.shape[2]
    for s, n in enumerate(b.lens):
        t = torch.arange(1000, n)
        ids = b.table[s, t // page].long()
        b.k[ids, :, t % page] = b.rows_kv[s][0][1000:]
    t = torch.arange(1000)
    b.k[b.prefix_table[0, t // page].long(), :, t % page] = b.rows_kv[0][0][:1000]
    o, lse = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("D,G", [(128, 1), (128, 4), (256, 16)])
@pytest.mark.parametrize("n", [4, 130, 641])
@pytest.mark.parametrize("shared", [False, True])
def test_drafted_values_that_are_not_finite(D, G, n, shared):
    """An infinity or a NaN in a drafted token's V reaches the rows that see it, in its channel, and no other; a NaN in its K
    every channel of those rows."""
    rows, P = 4, (n - 3) // 2 if shared else 0
    b = Batch([n, n + 9], [0, 2] if P else [0], [P] if P else [], rows, G, 1, D, 16, torch.bfloat16)
    page = 16
    clean = [sdp.fwd_cache16(**b.args())[0].clone()]
    assert sdp.poll_status() == sdp.SDP_OK

    def at(s, t):
        return int(b.table[s, t // page]), 0, t % page

    marks = [(0, n - 3, 5, math.inf), (0, n - 2, 100, math.nan), (1, n + 9 - 1, 64, -math.inf), (1, n + 9 - 3, D - 1, math.nan)]
    for s, t, c, x in marks:
        b.v[at(s, t)][c] = x
    o, lse = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK
    want = clean[0].clone()
    for s, t, c, x in marks:
        first = t - (b.lens[s] - rows)
        want[s, first:, :, c] = x
    same = (o == want) | (o.isnan() & want.isnan())
    assert same.all(), same.logical_not().nonzero()[:4]
    # the last token's key: its row alone
    for s, t, c, x in marks:
        b.v[at(s, t)][c] = 0.5
    before = sdp.fwd_cache16(**b.args())
    b.k[at(0, n - 1)][3] = math.nan
    o, lse = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK
    assert o[0, -1].isnan().all() and lse[0, -1].isnan().all()
    assert torch.equal(o[0, :-1], before[0][0, :-1]) and torch.equal(o[1], before[0][1])
    assert torch.equal(lse[0, :-1], before[1][0, :-1]) and torch.equal(lse[1], before[1][1])


def plain_batch(dtype=torch.bfloat16, **kw):
    a = dict(lens=[500, 300, 420, 290], cu=[0, 3], prefix=[280], rows=1, Hq=8, Hkv=2, D=128, page=32, dtype=dtype)
    a.update(kw)
    return Batch(**a)


@pytest.mark.gpu
def test_outputs_workspace_and_strided_tables():
    b = plain_batch()
    a = b.args()
    o, lse = sdp.fwd_cache16(**a)
    b.check(o, lse)
    # q without the row dimension; tables that are rows of wider ones
    wide = torch.full((4, a["block_table"].shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :-3] = a["block_table"]
    pwide = torch.full((1, a["prefix_table"].shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    pwide[:, :-5] = a["prefix_table"]
    need = sdp.cache16_workspace_bytes(4, 1, 8, 2, 128, torch.bfloat16, 1)
    for off in (0, 16):
        ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")[off:off + need]
        out, l2 = torch.full_like(o[:, 0], 9), torch.full_like(lse[:, 0], 9)
        got = sdp.fwd_cache16(**{**a, "q": a["q"][:, 0], "block_table": wide[:, :-3], "prefix_table": pwide[:, :-5]}, out=out, lse=l2,
                              workspace=ws)
        assert got[0] is out and got[1] is l2
        assert torch.equal(out, o[:, 0]) and torch.equal(l2, lse[:, 0])
    o2, none = sdp.fwd_cache16(**a, return_lse=False)
    assert none is None and torch.equal(o2, o)
    # one group of all
    b = plain_batch(lens=[500, 300, 420], cu=[0, 3])
    a = b.args()
    o, lse = sdp.fwd_cache16(**a)
    a["cu_groups"] = None
    o2, l2 = sdp.fwd_cache16(**a)
    assert torch.equal(o, o2) and torch.equal(lse, l2) and sdp.poll_status() == sdp.SDP_OK


@pytest.mark.gpu
def test_no_sequences():
    b = plain_batch()
    a = b.args()
    o, lse = sdp.fwd_cache16(a["q"][:0], a["cache"], a["cache_lens"][:0], a["block_table"][:0])
    assert o.shape == (0, 1, 8, 128) and lse.shape == (0, 1, 8)


@pytest.mark.gpu
def test_bad_lengths_groups_and_pages_are_reported():
    b = plain_batch()
    for key, at, x in (("cache_lens", 1, -1), ("cache_lens", 1, 32 * b.table.shape[1] + 1), ("cache_lens", 1, -2 ** 31),
                       ("cache_lens", 1, 2 ** 31 - 1)):
        a = b.args()
        a[key][at] = x
        out, lse = torch.full_like(a["q"], 3), torch.full(a["q"].shape[:3], 3.0, device="cuda")
        sdp.fwd_cache16(**a, out=out, lse=lse)
        assert sdp.poll_status() == sdp.SDP_ERR_BAD_SEQLENS
        assert (out[1] == 3).all() and (lse[1] == 3).all()  # as they were; the others are right
        b.check(out, lse, only=(0, 2, 3))
    full = plain_batch(own_pages=(0, 1, 2))  # every sequence's own pages are complete
    for key, at, x in (("prefix_lens", 0, -5), ("prefix_lens", 0, 32 * b.prefix_table.shape[1] + 1), ("cu_groups", 1, 5),
                       ("cu_groups", 0, -1), ("cu_groups", 0, 4)):
        a = full.args()
        a[key][at] = x
        o, lse = sdp.fwd_cache16(**a)
        assert sdp.poll_status() == sdp.SDP_ERR_BAD_SEQLENS
        full.check(o, lse)  # what is not shared is read from their own
    for key, at, x in (("block_table", (3, 2), -1), ("block_table", (0, 9), 1 << 30), ("prefix_table", (0, 1), 2 ** 31 - 1)):
        a = b.args()
        a[key][at] = x
        o, lse = sdp.fwd_cache16(**a)
        assert sdp.poll_status() == sdp.SDP_ERR_BAD_PAGES
        b.check(o, lse, only={"prefix_table": (3,)}.get(key, tuple(s for s in range(4) if s != at[0])))
    o, lse = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(o, lse)


@pytest.mark.gpu
def test_refusals_of_the_binding():
    b = plain_batch()
    good = b.args()
    q, c = good["q"], good["cache"]
    for kw in (dict(q=q.half()), dict(q=q.float()), dict(q=q[..., :64]), dict(q=q.cpu()), dict(q=q[0]), dict(q=q.transpose(0, 1)),
               dict(q=q.repeat(1, 40, 1, 1)), dict(q=torch.zeros(4, 1, 7, 128, device="cuda", dtype=q.dtype)),
               dict(cache=(c.k,)), dict(cache=sdp.Cache16(c.k, c.v.half())), dict(cache=sdp.Cache16(c.k, c.v[:, :, :16])),
               dict(cache_lens=good["cache_lens"].long()), dict(cache_lens=good["cache_lens"][:2]),
               dict(block_table=good["block_table"].long()), dict(block_table=good["block_table"][:2]),
               dict(block_table=good["block_table"].t()), dict(prefix_lens=None), dict(prefix_table=None),
               dict(prefix_lens=good["prefix_lens"].long()), dict(prefix_lens=good["prefix_lens"].repeat(2)),
               dict(cu_groups=good["cu_groups"][:1]), dict(cu_groups=good["cu_groups"].long()), dict(scale=math.nan),
               dict(out=q.half()), dict(out=q[:2]), dict(lse=torch.zeros(4, 8, device="cuda")), dict(stream="x"),
               dict(workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")), dict(q=q.clone().requires_grad_())):
        with pytest.raises((ValueError, sdp.SdpError)):
            sdp.fwd_cache16(**{**good, **kw})
    torch.cuda.synchronize()
    assert sdp.poll_status() == sdp.SDP_OK


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
def test_the_same_bits_each_time(D):
    b = plain_batch(lens=[3000, 2500, 2900, 100], prefix=[2400], rows=2, D=D)
    a = b.args()
    o, lse = sdp.fwd_cache16(**a)
    load = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(side):  # SMs that are taken for a while
            load = torch.tanh(load @ load)
        o2, l2 = sdp.fwd_cache16(**a)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert sdp.poll_status() == sdp.SDP_OK


@pytest.mark.gpu
def test_streams_and_two_graphs_at_once():
    bs = [plain_batch(seed=s, lens=[1500, 1300, 1420, 900 + s], prefix=[1280]) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in bs]
    graphs, outs = [], []
    for b, st in zip(bs, streams):
        a = b.args()
        torch.cuda.synchronize()
        ws = torch.empty(sdp.cache16_workspace_bytes(4, 1, 8, 2, 128, torch.bfloat16, 1), dtype=torch.uint8, device="cuda")
        want = sdp.fwd_cache16(**a, stream=st)
        st.synchronize()
        b.check(*want)
        out, lse = torch.zeros_like(a["q"]), torch.zeros(4, 1, 8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            sdp.fwd_cache16(**a, out=out, lse=lse, workspace=ws)
        graphs.append((g, a, ws))
        outs.append((out, lse, want))
    for _ in range(20):
        for (g, _, _), st, (out, lse, _) in zip(graphs, streams, outs):
            with torch.cuda.stream(st):
                out.zero_()
                lse.zero_()
                g.replay()
    torch.cuda.synchronize()
    assert sdp.poll_status() == sdp.SDP_OK
    for out, lse, want in outs:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
def test_waits_that_run_out(D):
    """No copy is issued: every wait gives up after its limit, the status says so, and the next call is right."""
    b = plain_batch(D=D)
    a = b.args()
    want = sdp.fwd_cache16(**a)
    assert sdp.poll_status() == sdp.SDP_OK
    old = sdp.set_wait_timeout_ms(20)
    sdp.set_debug_flags(1)
    try:
        sdp.fwd_cache16(**a)
        assert sdp.poll_status() == sdp.SDP_ERR_DEVICE_TIMEOUT
    finally:
        sdp.set_debug_flags(0)
        sdp.set_wait_timeout_ms(old)
    o, lse = sdp.fwd_cache16(**a)
    assert sdp.poll_status() == sdp.SDP_OK and torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_rows_past_32_bits_of_the_pool():
    """Pages whose first element lies beyond 2^32: written there and read there."""
    Hkv, page, D, n = 8, 128, 128, 300
    pages = (1 << 32) // (Hkv * page * D) + 40
    cache = sdp.Cache16(*(torch.empty(pages, Hkv, page, D, dtype=torch.float16, device="cuda") for _ in range(2)))
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(2 * n, Hkv, D, generator=g).half() for _ in range(2))
    table = torch.tensor([[pages - 1, pages - 30, pages - 7], [pages - 2, 0, pages - 9]], dtype=torch.int32)
    lens = torch.tensor([n, n], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    sdp.cache16_append(cache, k.cuda(), v.cuda(), cu, lens, table.cuda())
    b = Batch([n, n], [0], [], 1, 8, Hkv, D, page, torch.float16)
    b.rows_kv = [(k[:n], v[:n]), (k[n:], v[n:])]
    o, lse = sdp.fwd_cache16(b.q.cuda(), cache, lens, table.cuda())
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,D", [(1, 128), (3, 256)])
def test_a_captured_decoding_loop(dt, rows, D):
    """Prompts are appended once for the group and once a sequence; then one captured step appends each sequence's next tokens
    and attends over all of them, replayed while lengths grow. Every step against 64 bits, from what the cache holds."""
    dtype, Hq, Hkv, page, P, steps = DTYPES[dt], 8, 2, 16, 75, 9
    starts = [75, 83, 90, 75]
    nseq, most = len(starts), max(starts) + rows * steps
    g = torch.Generator().manual_seed(D + rows)
    per = -(-most // page)
    prefix_pages = -(-P // page)
    pool = nseq * per + prefix_pages
    order = torch.randperm(pool, generator=g).int()
    prefix_table = order[:prefix_pages][None].cuda()
    table = order[prefix_pages:].view(nseq, per).clone()
    table[:, :P // page] = order[:P // page]  # the prefix's full pages; the one that it ends in is each sequence's own
    table = table.cuda()
    cache = sdp.cache16_empty(pool, Hkv, D, page, dtype)
    rope = sdp.rope_table(sdp.rope_inv_freq(64), device="cuda")
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(dtype).cuda()

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def fused(tokens):
        return torch.randn(tokens, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()

    def parts(x):
        return dict(k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:])

    prompt = fused(P)
    sdp.cache16_append(cache, **parts(prompt), cu_seqlens=i32([0, P]), cache_lens=i32([P]), block_table=prefix_table, rope=rope, k_weight=w)
    own = [n - P for n in starts]
    rest = fused(sum(own))
    cu = i32([0, *torch.tensor(own).cumsum(0).tolist()])
    sdp.cache16_append(cache, **parts(rest), cu_seqlens=cu, cache_lens=i32(starts), block_table=table, rope=rope, k_weight=w)

    lens, x = i32(starts), fused(nseq * rows)
    cu_new = torch.arange(0, nseq * rows + 1, rows, dtype=torch.int32, device="cuda")
    plens = i32([P])
    out = torch.zeros(nseq, rows, Hq, D, dtype=dtype, device="cuda")
    lse = torch.zeros(nseq, rows, Hq, device="cuda")
    q_out = torch.zeros(nseq * rows, Hq, D, dtype=dtype, device="cuda")
    ws = torch.empty(sdp.cache16_workspace_bytes(nseq, rows, Hq, Hkv, D, dtype, 1), dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(rows)
        sdp.cache16_append(cache, **parts(x), cu_seqlens=cu_new, cache_lens=lens, block_table=table, rope=rope, q=x[:, :Hq], q_weight=w,
                           k_weight=w, q_out=q_out)
        sdp.fwd_cache16(q_out.view(nseq, rows, Hq, D), cache, lens, table, prefix_table, plens, out=out, lse=lse, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    b = Batch([1] * nseq, [0], [], rows, Hq, Hkv, D, page, dtype)
    for i in range(steps):
        x.copy_(fused(nseq * rows))
        graph.replay()
        assert sdp.poll_status() == sdp.SDP_OK
        b.lens = [n + rows * (i + 1) for n in starts]
        assert lens.tolist() == b.lens
        b.q = q_out.view(nseq, rows, Hq, D).cpu()
        b.rows_kv = []
        for s, n in enumerate(b.lens):
            t = torch.arange(n)
            ids = torch.where(t < P, prefix_table[0].cpu().long()[(t // page).clamp(max=prefix_pages - 1)], table[s].cpu().long()[t // page])
            b.rows_kv.append((cache.k.cpu()[ids, :, t % page], cache.v.cpu()[ids, :, t % page]))
            # the newest values are there as they came
            assert torch.equal(b.rows_kv[s][1][n - rows:], x[s * rows:(s + 1) * rows, Hq + Hkv:].cpu())
        b.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
def test_steps_that_follow_each_other_at_once(D):
    """Appends and attentions with nothing else between them, so that each is launched while the one before it ends, with one
    workspace for all: the bits of the same steps with a wait after each call."""
    Hq, Hkv, page, P, steps, dtype = 8, 2, 32, 400, 24, torch.bfloat16
    starts = [400, 640, 401, 1500]
    g = torch.Generator().manual_seed(D)
    per = -(-(max(starts) + steps) // page)
    table = torch.randperm(4 * per, generator=g).int().view(4, per)
    table[:, :P // page] = table[0, :P // page]
    ptable = table[:1, :-(-P // page)].contiguous().cuda()
    table = table.cuda()
    rope = sdp.rope_table(sdp.rope_inv_freq(D), device="cuda")
    first = (torch.randn(2, 4 * per, Hkv, page, D, generator=g) * 0.7).to(dtype).cuda()
    x = torch.randn(steps, 4, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()
    lens = [torch.tensor([n + i + 1 for n in starts], dtype=torch.int32, device="cuda") for i in range(steps)]
    cu = torch.arange(5, dtype=torch.int32, device="cuda")
    plens = torch.tensor([P], dtype=torch.int32, device="cuda")
    ws = torch.empty(sdp.cache16_workspace_bytes(4, 1, Hq, Hkv, D, dtype, 1), dtype=torch.uint8, device="cuda")
    results = []
    for wait in (True, False):
        cache = sdp.Cache16(first[0].clone(), first[1].clone())
        q = torch.zeros(steps, 4, Hq, D, dtype=dtype, device="cuda")
        o, lse = torch.zeros_like(q), torch.zeros(steps, 4, Hq, device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):
            sdp.cache16_append(cache, x[i, :, Hq:Hq + Hkv], x[i, :, Hq + Hkv:], cu, lens[i], table, rope=rope, q=x[i, :, :Hq], q_out=q[i])
            if wait:
                torch.cuda.synchronize()
            sdp.fwd_cache16(q[i], cache, lens[i], table, ptable, plens, out=o[i], lse=lse[i], workspace=ws)
            if wait:
                torch.cuda.synchronize()
        assert sdp.poll_status() == sdp.SDP_OK
        results.append((q, o, lse, cache.k, cache.v))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert not results[0][1].isnan().any()


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 48, 96, 160, 272, 1024, 4096])
@pytest.mark.parametrize("D", [128, 256])
def test_page_sizes(page, D):
    """Boxes of 16 to 128 keys, pages that tiles straddle and pages that hold many."""
    b = Batch([page + 5, 3 * page - 1, 2 * page, 700], [0, 3], [page - 3], 2, 6, 2, D, page, torch.float16)
    o, lse = sdp.fwd_cache16(**b.args())
    assert sdp.poll_status() == sdp.SDP_OK
    b.check(o, lse)


@pytest.mark.gpu
def test_several_host_threads():
    """Calls from threads of their own on streams of their own, workspaces from the allocator: each gets its own results."""
    import threading
    bs = [plain_batch(seed=s, lens=[700, 600 + s, 650], cu=[0, 3], prefix=[512]) for s in range(4)]
    args = [b.args() for b in bs]
    want = [tuple(t.clone() for t in sdp.fwd_cache16(**a)) for a in args]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(50):
                o, lse = sdp.fwd_cache16(**args[i])
                st.synchronize()
                if not (torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and sdp.poll_status() == sdp.SDP_OK
    for b, w in zip(bs, want):
        b.check(*w)
