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
