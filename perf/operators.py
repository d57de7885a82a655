"""The serving operators beside the attention forward, their plain forms, and the cases they are measured on.

Four operators of one serving path, each as a user's program calls it:

- ``rope``: the norm of every query and key head and the rotation by position, in one pass
  (``sdp.qk_norm_rope``), from a fused projection's strided rows into the layouts the attention reads;
- ``cache``: new tokens written into a paged cache held in 4 bits (``sdp.cache4_append``), and the
  sequences read back out of it as 16-bit rows for a prefill over them (``sdp.cache4_gather``);
- ``decode``: attention of each sequence's last tokens over that cache (``sdp.fwd_cache4``), over every
  key or over a sliding window with the first tokens kept visible;
- ``window``: the prefill attention with a sliding window and first tokens that stay visible
  (``sdp.fwd_window`` on dense batches, ``sdp.fwd_varlen_window`` on packed ones).

``run`` computes the plain form (elementary torch operations in 32 bits, angles in 64) where ``own`` is
false and calls the framework where it is true. ``exact`` is the definition in 64 bits, written apart.
"""
from __future__ import annotations

import itertools
import math
import random

import torch

own = False

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
GROUP = 64  # channels that share one scale and bias in the 4-bit cache


def listed():
    return [
        # one decode step of eight sequences: latency
        dict(name="rope_step8_d128", op="rope", B=0, T=8, Hq=32, Hkv=8, D=128, R=128, dtype="bf16", norm=True,
             interleaved=False, far=32768, base=10000.0, mscale=1.0),
        # a packed prefill batch of the headline head layout; a quarter of the head rotated, far positions
        dict(name="rope_prefill_d256", op="rope", B=0, T=39253, Hq=32, Hkv=2, D=256, R=64, dtype="fp16", norm=True,
             interleaved=False, far=1000000, base=5000000.0, mscale=1.0),
        # dense multi-head batch, interleaved pairs, rotation only, written [B, H, S, D] for the dense forward
        dict(name="rope_dense_b4_mha", op="rope", B=4, T=4099, Hq=32, Hkv=32, D=128, R=128, dtype="bf16", norm=False,
             interleaved=True, far=8192, base=10000.0, mscale=1.1),
        # one token each of 24 short sequences into their pages, and the sequences read back
        dict(name="cache_step24_d128", op="cache", nseq=24, lo=1, hi=200, new=1, Hkv=8, D=128, page=16, dtype="bf16",
             lens_seed=21),
        # twelve whole prompts written and read back (long-tailed lengths, headline head layout)
        dict(name="cache_prompts12_d256", op="cache", nseq=12, lo=256, hi=16384, new=0, Hkv=2, D=256, page=64,
             dtype="fp16", lens_seed=22),
        # a single sequence early in its answer: latency
        dict(name="decode_1x500_d128", op="decode", nseq=1, lo=500, hi=500, rows=1, Hq=32, Hkv=8, D=128, page=16,
             window=0, sinks=0, dtype="bf16", lens_seed=31),
        # eight long sequences, headline head layout
        dict(name="decode_8x16k_d256", op="decode", nseq=8, lo=16384, hi=16384, rows=1, Hq=32, Hkv=2, D=256, page=64,
             window=0, sinks=0, dtype="fp16", lens_seed=32),
        # a ragged batch with a window and four first tokens
        dict(name="decode_64_window4k_d128", op="decode", nseq=64, lo=128, hi=32768, rows=1, Hq=32, Hkv=8, D=128,
             page=64, window=4096, sinks=4, dtype="bf16", lens_seed=33),
        # four drafted tokens to verify on each of four long sequences
        dict(name="decode_4x32k_rows4_d128", op="decode", nseq=4, lo=30000, hi=32768, rows=4, Hq=32, Hkv=8, D=128,
             page=128, window=0, sinks=0, dtype="bf16", lens_seed=34),
        # the smallest dense prefill: latency
        dict(name="window_256_d128", op="window", B=1, nseq=0, lo=256, hi=256, past=0, Hq=4, Hkv=1, D=128, window=64,
             sinks=4, dtype="fp16", lens_seed=41),
        # twelve packed prompts of the headline head layout, a short window
        dict(name="window_varlen12_1k_d256", op="window", B=0, nseq=12, lo=256, hi=16384, past=0, Hq=32, Hkv=2, D=256,
             window=1024, sinks=4, dtype="fp16", lens_seed=42),
        # one long dense prompt, a wide window
        dict(name="window_16k_4k_d128", op="window", B=1, nseq=0, lo=16384, hi=16384, past=0, Hq=32, Hkv=8, D=128,
             window=4096, sinks=0, dtype="bf16", lens_seed=43),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "decode", "window"])
    D = rng.choice([128, 256])
    dtype = rng.choice(["fp16", "bf16"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 7, 8, 16] if Hkv <= 2 else [1, 2, 4])
    Hq = Hkv * G
    seed = rng.randrange(1 << 30)
    if op == "rope":
        B = rng.choice([0, 0, 1, 3])
        T = _log(rng, 1, 30000) if B == 0 else _log(rng, 1, 6000)
        R = rng.choice([0, 32, 64, 96, 128, D])
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, R=R, dtype=dtype, norm=R == 0 or rng.random() < 0.7,
                    interleaved=rng.random() < 0.5, far=_log(rng, 1000, 2000000),
                    base=rng.choice([10000.0, 500000.0, 5000000.0]), mscale=rng.choice([1.0, 1.0, 1.2]))
    if op == "cache":
        nseq = _log(rng, 1, 64)
        hi = _log(rng, 2, max(4, 40000 // nseq))
        return dict(op=op, nseq=nseq, lo=rng.choice([1, max(1, hi // 3)]), hi=hi, new=rng.choice([0, 1, 1, 5, 130]),
                    Hkv=Hkv, D=D, page=rng.choice([16, 32, 48, 64, 128, 256]), dtype=dtype, lens_seed=seed)
    if op == "decode":
        nseq = _log(rng, 1, 64)
        hi = _log(rng, 16, max(64, 160000 // nseq // (Hkv * D // 128)))
        return dict(op=op, nseq=nseq, lo=rng.choice([1, max(1, hi // 4)]), hi=hi, rows=rng.choice([1, 1, 1, 2, 5]),
                    Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 48, 64, 128, 256]),
                    window=rng.choice([0, 0, _log(rng, 1, hi)]), sinks=rng.choice([0, 1, 4, 33]), dtype=dtype,
                    lens_seed=seed)
    B = rng.choice([0, 0, 0, 1, 2, 3])
    nseq = 0 if B else _log(rng, 1, 16)
    Hq, Hkv = (Hq, Hkv) if Hq <= 16 else (16, 1)
    W = _log(rng, 16, 3000)
    most = min(30000, int(9e11 / (4 * (W + 64) * Hq * D))) // max(B, nseq)  # rows of a sequence
    hi = _log(rng, 64, min(8192, max(65, most)))
    return dict(op="window", B=B, nseq=nseq, lo=hi if B else rng.choice([1, max(1, hi // 4)]), hi=hi,
                past=rng.choice([0, _log(rng, 1, 1000)]) if B else 0, Hq=Hq, Hkv=Hkv, D=D, window=W,
                sinks=rng.choice([0, 1, 4, 40]), dtype=dtype, lens_seed=seed)


def _lens(case):
    """The sequence lengths of a case, from its own numbers: log-uniform in [lo, hi]."""
    r = random.Random(case["lens_seed"])
    return [_log(r, case["lo"], case["hi"]) for _ in range(max(1, case["nseq"]))]


def _offsets(lens):
    return [0, *itertools.accumulate(lens)]


def _cuda():
    return torch.device("cuda", torch.cuda.current_device())


def _normal(g, *shape):
    return torch.randn(*shape, device=g.device, generator=g)


def _keys(g, *shape):
    """Key-like rows: unit normal with a few loud channels and an offset on others, as projections give."""
    x = _normal(g, *shape)
    gain = 1 + 3 * (torch.rand(shape[-1], device=g.device, generator=g) < 0.03).float()
    return x * gain + 0.5 * _normal(g, shape[-1])


def _inv_freq(case, device):
    i = torch.arange(case["R"] // 2, dtype=torch.float64, device=device)
    return torch.exp(-math.log(case["base"]) * 2 * i / max(1, case["R"]))


def _pages(case, lens, g):
    """A block table that scatters each sequence's pages over the pool, and the pool's page count."""
    need = [-(-n // case["page"]) for n in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, device=g.device, generator=g).int()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=g.device)
    for s, first in enumerate(_offsets(need)[:-1]):
        table[s, :need[s]] = order[first:first + need[s]]
    return table, pool


def _slots(case, lens, table):
    """Page and place in the page of every token of every sequence, packed back to back."""
    n = torch.tensor(lens, device=table.device)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=table.device), n)
    first = torch.cumsum(n, 0) - n
    pos = torch.arange(int(sum(lens)), device=table.device) - first[seq]
    return table[seq, pos // case["page"]].long(), pos % case["page"], seq, pos


def _empty_cache(case, pool, device):
    shape = (pool, case["Hkv"], case["page"])
    codes = [torch.zeros(*shape, case["D"] // 2, dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.zeros(*shape, case["D"] // GROUP, 2, dtype=torch.bfloat16, device=device) for _ in range(2)]
    return [codes[0], scales[0], codes[1], scales[1]]


def prepare(case, seed):
    dev = _cuda()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)
    op, dt, D = case["op"], DT[case["dtype"]], case["D"]
    st = dict(case=case)
    if op == "rope":
        Hq, Hkv, T, B = case["Hq"], case["Hkv"], case["T"], max(1, case["B"])
        qkv = _normal(g, B * T, (Hq + 2 * Hkv) * D).to(dt)  # the fused projection's output
        q = qkv[:, :Hq * D].view(B, T, Hq, D)
        k = qkv[:, Hq * D:(Hq + Hkv) * D].view(B, T, Hkv, D)
        start = torch.randint(0, max(1, case["far"] - T), (B, 1), device=dev, generator=g)
        if case["B"] == 0:
            st["q"], st["k"] = q[0], k[0]
            # a packed batch: runs of consecutive positions, each sequence with a start of its own
            run = torch.arange(T, device=dev) // 1000
            starts = torch.randint(0, max(1, case["far"] - 1000), (T // 1000 + 1,), device=dev, generator=g)
            st["positions"] = (starts[run] + torch.arange(T, device=dev) % 1000).int()
        else:
            st["q"], st["k"] = q.transpose(1, 2), k.transpose(1, 2)
            st["positions"] = (start + torch.arange(T, device=dev)).int()
        st["wq"] = (1 + 0.2 * _normal(g, D)).to(dt) if case["norm"] else None
        st["wk"] = (1 + 0.2 * _normal(g, D)).to(dt) if case["norm"] else None
        st["inv_freq"] = _inv_freq(case, dev)
        if own:
            import gqa_flash_attention_gb300 as sdp
            st["table"] = sdp.rope_table(st["inv_freq"], mscale=case["mscale"]) if case["R"] else None
    elif op == "cache":
        lens = _lens(case)
        new = [n if case["new"] == 0 else min(n, case["new"]) for n in lens]
        table, pool = _pages(case, lens, g)
        st["parts"] = _empty_cache(case, pool, dev)
        page, place, _, _ = _slots(case, lens, table)
        total = int(sum(lens))
        _store(st["parts"], page, place, _keys(g, total, case["Hkv"], D).to(dt), _normal(g, total, case["Hkv"], D).to(dt))
        st["k"] = _keys(g, int(sum(new)), case["Hkv"], D).to(dt)
        st["v"] = _normal(g, int(sum(new)), case["Hkv"], D).to(dt)
        st["table"], st["total"] = table, total
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        st["cu_new"] = torch.tensor(_offsets(new), dtype=torch.int32, device=dev)
        st["cu"] = torch.tensor(_offsets(lens), dtype=torch.int32, device=dev)
    elif op == "decode":
        lens = _lens(case)
        table, pool = _pages(case, lens, g)
        st["parts"] = _empty_cache(case, pool, dev)
        page, place, _, _ = _slots(case, lens, table)
        step = max(1, (1 << 28) // (case["Hkv"] * D))
        for a in range(0, len(page), step):
            n = min(step, len(page) - a)
            _store(st["parts"], page[a:a + n], place[a:a + n], _keys(g, n, case["Hkv"], D).to(dt),
                   _normal(g, n, case["Hkv"], D).to(dt))
        st["q"] = _normal(g, len(lens), case["rows"], case["Hq"], D).to(dt)
        st["table"], st["max_len"] = table, max(lens)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    else:
        lens = _lens(case)
        if case["B"]:
            S = lens[0]
            st["q"] = _normal(g, case["B"], case["Hq"], S, D).to(dt)
            st["k"] = _keys(g, case["B"], case["Hkv"], S + case["past"], D).to(dt)
            st["v"] = _normal(g, case["B"], case["Hkv"], S + case["past"], D).to(dt)
        else:
            T = int(sum(lens))
            st["q"] = _normal(g, T, case["Hq"], D).to(dt)
            st["k"] = _keys(g, T, case["Hkv"], D).to(dt)
            st["v"] = _normal(g, T, case["Hkv"], D).to(dt)
            st["cu"] = torch.tensor(_offsets(lens), dtype=torch.int32, device=dev)
            st["max_len"] = max(lens)
    if own and op in ("cache", "decode"):
        import gqa_flash_attention_gb300 as sdp
        st["cache"] = sdp.Cache4(*st["parts"])
    return st


# ------------------------------------------------------------------ plain forms


def _norm(x, w):
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return y * w.float()


def _rotate(x, cos, sin, R, interleaved):
    """The first R channels of x turned by the angles of its row; cos and sin broadcast against [..., R / 2]."""
    rot, rest = x[..., :R], x[..., R:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = rot[..., :R // 2], rot[..., R // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1)


def _plain_rope(st):
    c = st["case"]
    angle = st["positions"].double().unsqueeze(-1) * st["inv_freq"]
    cos, sin = (torch.cos(angle) * c["mscale"]).float(), (torch.sin(angle) * c["mscale"]).float()
    # a head axis: [T, 1, R/2] beside [T, H, D], or [B, 1, S, R/2] beside [B, H, S, D]
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    q, k = st["q"].float(), st["k"].float()
    if c["norm"]:
        q, k = _norm(q, st["wq"]), _norm(k, st["wk"])
    q, k = _rotate(q, cos, sin, c["R"], c["interleaved"]), _rotate(k, cos, sin, c["R"], c["interleaved"])
    return q.to(st["q"].dtype), k.to(st["k"].dtype)


def _quantise(x):
    """Codes (two to a byte, the lower channel low) and (scale, bias) of [..., D] rows in groups of 64 channels."""
    x = x.float().unflatten(-1, (-1, GROUP))
    bias = x.amin(-1).bfloat16()
    span = x.amax(-1) - bias.float()
    scale = (span / torch.full_like(span, 15)).clamp_min(0).bfloat16()  # (a number there would be inverted first)
    step = torch.where(scale > 0, scale.float(), torch.ones_like(scale, dtype=torch.float32)).unsqueeze(-1)
    # (x - bias) / scale often lies on a border between two codes: divided, not multiplied by an inverse
    code = torch.round((x - bias.float().unsqueeze(-1)) / step).clamp(0, 15).to(torch.uint8)
    code = torch.where((scale > 0).unsqueeze(-1), code, torch.zeros_like(code)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.stack((scale, bias), -1)


def _store(parts, page, place, k, v):
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    parts[0][page, :, place], parts[1][page, :, place] = kc, ks
    parts[2][page, :, place], parts[3][page, :, place] = vc, vs


def _values(codes, scales):
    """fp32 rows [..., D] from codes [..., D / 2] and (scale, bias) [..., D / 64, 2]."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    s = scales.float()
    return (code * s[..., :1] + s[..., 1:]).flatten(-2)


def _plain_cache(st):
    c, parts = st["case"], st["parts"]
    n = (st["cu_new"][1:] - st["cu_new"][:-1]).long()
    rows = st["k"].shape[0]
    seq = torch.repeat_interleave(torch.arange(len(n), device=n.device), n, output_size=rows)
    pos = torch.arange(rows, device=n.device) - st["cu_new"][seq] + (st["lens"][seq] - n[seq])
    _store(parts, st["table"][seq, pos // c["page"]].long(), pos % c["page"], st["k"], st["v"])
    m = st["lens"].long()
    seq = torch.repeat_interleave(torch.arange(len(m), device=m.device), m, output_size=st["total"])
    pos = torch.arange(st["total"], device=m.device) - st["cu"][seq]
    page, place = st["table"][seq, pos // c["page"]].long(), pos % c["page"]
    k = _values(parts[0][page, :, place], parts[1][page, :, place])
    v = _values(parts[2][page, :, place], parts[3][page, :, place])
    return k.to(st["k"].dtype), v.to(st["v"].dtype)


def _softmax(s, v_of):
    """(weights applied by v_of, natural log-sum-exp) of scores [..., keys]; a row without keys gives 0 and -inf."""
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(m.isinf(), torch.zeros_like(m), m))
    l = e.sum(-1, keepdim=True)
    o = v_of(e) / torch.where(l > 0, l, torch.ones_like(l)).squeeze(-1).unsqueeze(-1)
    return o, torch.log(l.squeeze(-1)) + torch.where(m.isinf(), torch.zeros_like(m), m).squeeze(-1)


def _plain_decode(st):
    c, parts = st["case"], st["parts"]
    G, n, L = c["Hq"] // c["Hkv"], c["rows"], st["max_len"]
    j = torch.arange(L, device=st["q"].device)
    page = st["table"][:, j // c["page"]].clamp_min(0).long()  # [nseq, L]
    place = (j % c["page"]).expand_as(page)
    k = _values(parts[0][page, :, place], parts[1][page, :, place])  # [nseq, L, Hkv, D]
    v = _values(parts[2][page, :, place], parts[3][page, :, place])
    q = st["q"].float().unflatten(2, (c["Hkv"], G))  # [nseq, n, Hkv, G, D]
    s = torch.einsum("bngid,bkgd->bngik", q, k) / math.sqrt(c["D"])
    p = st["lens"].unsqueeze(1) - n + torch.arange(n, device=j.device)  # [nseq, n] positions of the rows
    seen = (j <= p.unsqueeze(-1)) & (j < st["lens"].view(-1, 1, 1))
    if c["window"]:
        seen = seen & ((j > p.unsqueeze(-1) - c["window"]) | (j < c["sinks"]))
    s = s.masked_fill(~seen[:, :, None, None], -math.inf)
    o, lse = _softmax(s, lambda e: torch.einsum("bngik,bkgd->bngid", e, v))
    return o.flatten(2, 3).to(st["q"].dtype), lse.flatten(2, 3)


def _plain_window(st):
    c = st["case"]
    G, W, S = c["Hq"] // c["Hkv"], c["window"], c["sinks"]
    if c["B"]:  # the batch as packed sequences
        B, H, Sq, D = st["q"].shape
        q, k, v = (st[x].transpose(1, 2).flatten(0, 1) for x in "qkv")
        nq = torch.full((B,), Sq, device=q.device)
        nk = torch.full((B,), Sq + c["past"], device=q.device)
    else:
        q, k, v = st["q"], st["k"], st["v"]
        nq = nk = (st["cu"][1:] - st["cu"][:-1]).long()
    T = q.shape[0]
    seq = torch.repeat_interleave(torch.arange(len(nq), device=q.device), nq, output_size=T)
    base = (torch.cumsum(nk, 0) - nk)[seq]  # first key row of a query's sequence
    at = torch.arange(T, device=q.device) - (torch.cumsum(nq, 0) - nq)[seq] + (nk - nq)[seq] + base  # its own key row
    # Query blocks of BQ packed rows; a block's keys run from W - 1 before its first row's own key to its last row's.
    # (A block that straddles two sequences of different pasts has its rows' keys further apart: `past` more rows each.)
    BQ = max(64, W // 4)
    nb = -(-T // BQ)
    pad = nb * BQ - T
    cut = lambda x: torch.cat((x, x[-1:].expand(pad, *x.shape[1:]))).unflatten(0, (nb, BQ))  # noqa: E731
    at_b, base_b = cut(at), cut(base)
    span = BQ + W - 1 + c["past"] * (BQ // max(1, T // len(nq)) + 1) * (len(nq) > 1)
    rows = at_b[:, :1] - W + 1 + torch.arange(span, device=q.device)  # [nb, span]
    kb, vb = (x[rows.clamp(0, k.shape[0] - 1)].float() for x in (k, v))  # [nb, span, Hkv, D]
    qb = cut(q.float()).unflatten(2, (c["Hkv"], G))  # [nb, BQ, Hkv, G, D]
    s = torch.einsum("bqgid,bkgd->bgiqk", qb, kb)
    r = rows.unsqueeze(1)
    seen = (r <= at_b.unsqueeze(-1)) & (r > at_b.unsqueeze(-1) - W) & (r >= base_b.unsqueeze(-1)) & (r < k.shape[0])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    # the first S keys of each row's sequence, where the window does not hold them already
    first = base.unsqueeze(1) + torch.arange(S, device=q.device)  # [T, S]
    ks, vs = (x[first.clamp(0, k.shape[0] - 1)].float() for x in (k, v))  # [T, S, Hkv, D]
    s0 = torch.einsum("tgid,tsgd->tgis", q.float().unflatten(1, (c["Hkv"], G)), ks)
    s0 = s0.masked_fill(~(first <= (at - W).unsqueeze(1))[:, None, None], -math.inf)
    s0 = cut(s0).permute(0, 2, 3, 1, 4)  # [nb, Hkv, G, BQ, S]
    vs = cut(vs)

    def weigh(e):
        return (torch.einsum("bgiqk,bkgd->bgiqd", e[..., :span], vb)
                + torch.einsum("bgiqs,bqsgd->bgiqd", e[..., span:], vs))

    o, lse = _softmax(torch.cat((s, s0), -1) / math.sqrt(c["D"]), weigh)
    o = o.permute(0, 3, 1, 2, 4).flatten(0, 1).flatten(1, 2)[:T].to(q.dtype)  # [T, Hq, D]
    lse = lse.permute(0, 3, 1, 2).flatten(0, 1).flatten(1, 2)[:T]  # [T, Hq]
    if c["B"]:
        return o.unflatten(0, (B, Sq)).transpose(1, 2).contiguous(), lse.unflatten(0, (B, Sq)).transpose(1, 2).contiguous()
    return o, lse.t().contiguous()


def run(state):
    c = state["case"]
    if not own:
        return {"rope": _plain_rope, "cache": _plain_cache, "decode": _plain_decode, "window": _plain_window}[c["op"]](state)
    import gqa_flash_attention_gb300 as sdp
    if c["op"] == "rope":
        return sdp.qk_norm_rope(state["q"], state["k"], state["positions"], state["table"], q_weight=state["wq"],
                                k_weight=state["wk"], eps=1e-6, interleaved=c["interleaved"])
    if c["op"] == "cache":
        sdp.cache4_append(state["cache"], state["k"], state["v"], state["cu_new"], state["lens"], state["table"])
        return sdp.cache4_gather(state["cache"], state["cu"], state["table"], state["total"], dtype=state["k"].dtype)
    if c["op"] == "decode":
        return sdp.fwd_cache4(state["q"], state["cache"], state["lens"], state["table"], window=c["window"],
                              sinks=c["sinks"])
    if c["B"]:
        return sdp.fwd_window(state["q"], state["k"], state["v"], c["window"], sinks=c["sinks"])
    return sdp.fwd_varlen_window(state["q"], state["k"], state["v"], state["cu"], state["cu"], state["max_len"],
                                 c["window"], sinks=c["sinks"])


# ------------------------------------------------------------------ what a pass cannot do without


def _seen(c, lens):
    """Keys seen, summed over the query rows of one head, and the distinct keys that some row sees."""
    pairs = keys = 0
    W, S = c["window"], c["sinks"]
    for n in lens:
        q = n if c["op"] == "window" else min(n, c["rows"])
        n = n + (c["past"] if c["op"] == "window" else 0)
        first = n - q  # position of the first row
        if W == 0:
            pairs += sum(range(first + 1, n + 1))
            keys += n
            continue
        full = max(0, min(q, W - first))  # rows with fewer than W keys before and at them
        pairs += sum(range(first + 1, first + full + 1)) + (q - full) * W
        pairs += sum(min(S, max(0, p + 1 - W)) for p in range(first, n)) if S else 0
        lo = max(0, first - W + 1)
        keys += n - lo + min(S, lo)
    return pairs, keys


def work(case):
    c, D = case, case["D"]
    if c["op"] == "rope":
        rows = max(1, c["B"]) * c["T"]
        heads = c["Hq"] + c["Hkv"]
        w = 4 * D if c["norm"] else 0
        return {"bytes": rows * heads * D * 4 + rows * 4 + w + c["R"] * 4,
                "flops": rows * heads * ((4 * D if c["norm"] else 0) + 3 * c["R"])}
    row4 = D // 2 + D // GROUP * 4  # one head's row in the cache
    lens = _lens(c)
    if c["op"] == "cache":
        new = sum(n if c["new"] == 0 else min(n, c["new"]) for n in lens)
        total = sum(lens)
        pages = sum(-(-n // c["page"]) for n in lens)
        # append: the new 16-bit rows in, their codes and scales out; gather: every row's codes in, 16 bits out
        return {"bytes": 2 * c["Hkv"] * (new * (2 * D + row4) + total * (row4 + 2 * D)) + 2 * 4 * pages + 16 * len(lens),
                "flops": 2 * c["Hkv"] * D * (5 * new + 2 * total)}
    pairs, keys = _seen(c, lens)
    if c["op"] == "decode":
        rows = len(lens) * c["rows"]
        return {"bytes": 2 * c["Hkv"] * keys * row4 + rows * c["Hq"] * (4 * D + 4) + 4 * len(lens) + 4 * keys // c["page"],
                "flops": 4 * D * c["Hq"] * pairs}
    b = max(1, c["B"])
    tq, tk = b * sum(lens), b * (sum(lens) + c["past"] * len(lens))
    return {"bytes": tq * c["Hq"] * (4 * D + 4) + tk * c["Hkv"] * 4 * D, "flops": 4 * D * c["Hq"] * pairs * b}


# ------------------------------------------------------------------ the definitions in 64 bits


def _turn(x, pos, freq, R, interleaved, mscale):
    """Rows x [n, H, D] (64 bits) at positions pos [n]: channel pairs as complex numbers times exp(i pos f)."""
    ang = pos.double()[:, None] * freq[None]
    z = torch.polar(torch.full_like(ang, mscale), ang)[:, None]
    pairs = x[..., :R].reshape(*x.shape[:-1], R // 2, 2) if interleaved else torch.stack((x[..., :R // 2], x[..., R // 2:R]), -1)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    y = y.flatten(-2) if interleaved else torch.cat((y[..., 0], y[..., 1]), -1)
    return torch.cat((y, x[..., R:]), -1)


def _attend(q, k, v, pos, window, sinks, scale):
    """q [n, H, D], k and v [m, Hkv, D] in 64 bits, pos [n]: rows see keys 0..pos (of the window or the first ones)."""
    n, H, D = q.shape
    G = H // k.shape[1]
    o = torch.zeros(n, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    for a in range(0, n, 512):
        p = pos[a:a + 512]
        hi = int(p.max()) + 1
        if hi <= 0:
            continue
        lo = max(0, int(p.min()) - window + 1) if window else 0
        keys = torch.arange(hi, device=q.device)
        keys = keys[(keys >= lo) | (keys < sinks)]
        keys = keys[keys < k.shape[0]]
        ok = keys[None] <= p[:, None]
        if window:
            ok &= (keys[None] > p[:, None] - window) | (keys[None] < sinks)
        kk, vv = k[keys].transpose(0, 1), v[keys].transpose(0, 1)  # [Hkv, m, D]
        qq = q[a:a + 512].transpose(0, 1).reshape(k.shape[1], -1, D)  # [Hkv, G * rows, D]
        s = (qq @ kk.transpose(1, 2)) * scale
        s = s.view(k.shape[1], G, -1, len(keys)).masked_fill(~ok, -math.inf)
        l = torch.logsumexp(s, -1)
        w = torch.exp(s - torch.where(l.isinf(), torch.zeros_like(l), l)[..., None])
        o[a:a + 512] = (w.flatten(1, 2) @ vv).view(H, -1, D).transpose(0, 1)
        lse[a:a + 512] = l.flatten(0, 1).t()
    return o, lse


def _read(parts, which, page, place):
    b = parts[2 * which][page, :, place].to(torch.int64)
    s = parts[2 * which + 1][page, :, place].double()
    x = torch.empty(*b.shape[:-1], b.shape[-1] * 2, dtype=torch.float64, device=b.device)
    x[..., 0::2], x[..., 1::2] = (b % 16).double(), torch.div(b, 16, rounding_mode="floor").double()
    return x * s[..., 0].repeat_interleave(GROUP, -1) + s[..., 1].repeat_interleave(GROUP, -1)


def _held(x):
    """The values that 4-bit codes with their rounded scale and bias stand for, of 64-bit rows."""
    y = torch.empty_like(x)
    for a in range(0, x.shape[-1], GROUP):
        part = x[..., a:a + GROUP]
        low = part.amin(-1, keepdim=True).to(torch.bfloat16).double()
        span = part.amax(-1, keepdim=True) - low
        step = (span / torch.full_like(span, 15)).clamp_min(0).to(torch.bfloat16).double()
        code = torch.where(step > 0, torch.round((part - low) / step.clamp_min(1e-300)), torch.zeros_like(part)).clamp(0, 15)
        y[..., a:a + GROUP] = low + step * code
    return y


def exact(case, seed):
    global own
    was, own = own, False
    st = prepare(case, seed)
    own = was
    c = case
    if c["op"] == "rope":
        out = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            rows = x.transpose(1, 2).reshape(-1, x.shape[1], c["D"]) if c["B"] else x
            if rows.numel() > 1 << 29:
                return None
            y = rows.double()
            if c["norm"]:
                y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / c["D"] + 1e-6) * w.double()
            if c["R"]:
                y = _turn(y, st["positions"].reshape(-1), st["inv_freq"], c["R"], c["interleaved"], c["mscale"])
            out.append(y.view(c["B"], c["T"], -1, c["D"]).transpose(1, 2).contiguous() if c["B"] else y)
        return tuple(out)
    lens = _lens(c)
    if c["op"] == "cache":
        page, place, seq, pos = _slots(c, lens, st["table"])
        out = []
        cu_new, cu = st["cu_new"].tolist(), st["cu"].tolist()
        for which, x in ((0, st["k"]), (1, st["v"])):
            y = _read(st["parts"], which, page, place)
            h = _held(x.double())
            for s in range(len(lens)):
                n = cu_new[s + 1] - cu_new[s]
                y[cu[s + 1] - n:cu[s + 1]] = h[cu_new[s]:cu_new[s + 1]]
            out.append(y)
        return tuple(out)
    scale = 1 / math.sqrt(c["D"])
    if c["op"] == "decode":
        page, place, _, _ = _slots(c, lens, st["table"])
        os_, ls, a = [], [], 0
        for s, n in enumerate(lens):
            k, v = (_read(st["parts"], w, page[a:a + n], place[a:a + n]) for w in (0, 1))
            pos = torch.arange(n - c["rows"], n, device=k.device)
            o, l = _attend(st["q"][s].double(), k, v, pos, c["window"], c["sinks"], scale)
            os_.append(o)
            ls.append(l)
            a += n
        return torch.stack(os_), torch.stack(ls)
    os_, ls = [], []
    if c["B"]:
        for b in range(c["B"]):
            q, k, v = (st[x][b].transpose(0, 1).double() for x in "qkv")
            pos = torch.arange(k.shape[0] - q.shape[0], k.shape[0], device=q.device)
            o, l = _attend(q, k, v, pos, c["window"], c["sinks"], scale)
            os_.append(o.transpose(0, 1))
            ls.append(l.t())
        return torch.stack(os_).contiguous(), torch.stack(ls).contiguous()
    cu = st["cu"].tolist()
    for s, n in enumerate(lens):
        q, k, v = (st[x][cu[s]:cu[s + 1]].double() for x in "qkv")
        o, l = _attend(q, k, v, torch.arange(n, device=q.device), c["window"], c["sinks"], scale)
        os_.append(o)
        ls.append(l)
    return torch.cat(os_), torch.cat(ls).t().contiguous()
