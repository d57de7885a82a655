"""The 16-bit paged cache's operators, their plain forms, and the cases they are measured on.

Two operators of one decoding path, each as a user's program calls it:

- ``append``: new tokens' keys and values into a paged cache of 16-bit rows, norms and position rotation of
  the queries and keys applied on the way (``sdp.cache16_append``), from a fused projection's strided rows;
- ``shared``: attention of each sequence's last tokens over that cache, for batches whose sequences share
  prefixes that are read and multiplied once for all of a group (``sdp.fwd_cache16``), or share none.

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


def listed():
    return [
        # one decode step of eight sequences: latency
        dict(name="append_step8_d128", op="append", nseq=8, lo=20, hi=500, new=1, Hq=32, Hkv=8, D=128, R=128, page=16,
             dtype="bf16", norm=True, interleaved=False, base=10000.0, mscale=1.0, far=0, lens_seed=11),
        # twelve whole prompts of the headline head layout, a quarter of the head rotated
        dict(name="append_prompts12_d256", op="append", nseq=12, lo=256, hi=16384, new=0, Hq=32, Hkv=2, D=256, R=64,
             page=64, dtype="fp16", norm=True, interleaved=False, base=5000000.0, mscale=1.0, far=0, lens_seed=12),
        # a chunk of each of 24 prompts, multi-head, interleaved pairs, rotation only, positions of the caller's own
        dict(name="append_chunks24_mha", op="append", nseq=24, lo=100, hi=3000, new=130, Hq=32, Hkv=32, D=128, R=128,
             page=48, dtype="bf16", norm=False, interleaved=True, base=10000.0, mscale=1.1, far=1000000, lens_seed=13),
        # four answers to one short prompt: latency
        dict(name="shared_4x500_d128", op="shared", nseq=4, groups=1, plo=500, phi=500, lo=1, hi=60, rows=1, Hq=32,
             Hkv=8, D=128, page=16, whole=False, dtype="bf16", lens_seed=21),
        # 64 conversations behind one instruction prompt
        dict(name="shared_64x8k_d128", op="shared", nseq=64, groups=1, plo=8192, phi=8192, lo=10, hi=2000, rows=1,
             Hq=32, Hkv=8, D=128, page=64, whole=True, dtype="bf16", lens_seed=22),
        # 256 samples of one long prompt, headline head layout: the prefix is a matrix product
        dict(name="shared_256x16k_d256", op="shared", nseq=256, groups=1, plo=16384, phi=16384, lo=16, hi=512, rows=1,
             Hq=32, Hkv=2, D=256, page=64, whole=True, dtype="fp16", lens_seed=23),
        # four prompts of different lengths, four drafted tokens to verify on each of their answers
        dict(name="shared_groups4_rows4_d128", op="shared", nseq=60, groups=4, plo=1500, phi=12000, lo=20, hi=3500,
             rows=4, Hq=32, Hkv=8, D=128, page=128, whole=True, dtype="bf16", lens_seed=24),
        # multi-head: one row a head and sequence, a prefix that ends inside a page
        dict(name="shared_32x4k_mha", op="shared", nseq=32, groups=1, plo=4001, phi=4001, lo=1, hi=300, rows=1, Hq=32,
             Hkv=32, D=128, page=32, whole=False, dtype="fp16", lens_seed=25),
        # no prefix: plain decoding of eight long sequences, headline head layout
        dict(name="alone_8x16k_d256", op="shared", nseq=8, groups=0, plo=0, phi=0, lo=16384, hi=16384, rows=1, Hq=32,
             Hkv=2, D=256, page=64, whole=True, dtype="fp16", lens_seed=26),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "shared", "shared"])
    D = rng.choice([128, 256])
    dtype = rng.choice(["fp16", "bf16"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 7, 8, 16] if Hkv <= 2 else [1, 2, 4])
    Hq = Hkv * G
    page = rng.choice([16, 32, 48, 64, 128, 256])
    seed = rng.randrange(1 << 30)
    if op == "append":
        nseq = _log(rng, 1, 256)
        hi = _log(rng, 2, max(4, 40000 // nseq))
        R = rng.choice([0, 32, 64, 96, 128, D])
        return dict(op=op, nseq=nseq, lo=rng.choice([1, max(1, hi // 3)]), hi=hi, new=rng.choice([0, 1, 1, 5, 130]),
                    Hq=Hq, Hkv=Hkv, D=D, R=R, page=page, dtype=dtype, norm=R == 0 or rng.random() < 0.7,
                    interleaved=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0, 5000000.0]),
                    mscale=rng.choice([1.0, 1.0, 1.2]), far=rng.choice([0, 0, 2000000]), lens_seed=seed)
    nseq = _log(rng, 1, 256)
    rows = rng.choice([1, 1, 1, 2, 5])
    groups = rng.choice([0, 1, 1, 1, min(nseq, 3)])
    # at most about a tenth of a TFLOP over the prefixes, and half a GB of keys and values behind them
    row_bytes = 4 * Hkv * D
    phi = _log(rng, 16, max(17, min(32768, int(1e11 / (4 * D * Hq * nseq * rows))))) if groups else 0
    hi = _log(rng, 8, max(9, min(16384, 500000000 // row_bytes // nseq)))
    if groups == 0:
        hi = max(hi, rows)
    return dict(op=op, nseq=nseq, groups=groups, plo=max(1, phi // 3) if groups > 1 else phi, phi=phi,
                lo=rng.choice([1, max(1, hi // 4)]), hi=hi, rows=rows, Hq=Hq, Hkv=Hkv, D=D, page=page,
                whole=rng.random() < 0.6, dtype=dtype, lens_seed=seed)


def _offsets(lens):
    return [0, *itertools.accumulate(lens)]


def _lens(case):
    """The sequence lengths of an append case: log-uniform in [lo, hi], the new tokens among them."""
    r = random.Random(case["lens_seed"])
    return [_log(r, case["lo"], case["hi"]) for _ in range(case["nseq"])]


def _new(case, lens):
    return [n if case["new"] == 0 else min(n, case["new"]) for n in lens]


def _batch(case):
    """A shared case's group of each sequence (-1: none), group offsets, prefix lengths and whole lengths."""
    r = random.Random(case["lens_seed"])
    n, k = case["nseq"], case["groups"]
    cu = [0, *sorted(r.randint(0, n) for _ in range(k - 1)), n] if k else [0]
    prefix = [_log(r, case["plo"], case["phi"]) for _ in range(k)]
    if case["whole"]:
        prefix = [max(p // case["page"], 1) * case["page"] for p in prefix]
    group = [g for g in range(k) for _ in range(cu[g + 1] - cu[g])] if k else [-1] * n
    lens = [max(case["rows"], _log(r, case["lo"], case["hi"])) + (prefix[g] if g >= 0 else 0) for g in group]
    return group, cu, prefix, lens


def _cuda():
    return torch.device("cuda", torch.cuda.current_device())


def _normal(g, *shape):
    return torch.randn(*shape, device=g.device, generator=g)


def _keys(g, *shape):
    """Key-like rows: unit normal with a few loud channels and an offset on others, as projections give."""
    x = _normal(g, *shape)
    gain = 1 + 3 * (torch.rand(shape[-1], device=g.device, generator=g) < 0.03).float()
    return x * gain + 0.5 * _normal(g, shape[-1])


def _int32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = _cuda()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 29)
    dt, D, Hq, Hkv, page = DT[case["dtype"]], case["D"], case["Hq"], case["Hkv"], case["page"]
    st = dict(case=case)
    if case["op"] == "append":
        lens = _lens(case)
        new = _new(case, lens)
        need = [-(-n // page) for n in lens]
        pool = sum(need) + 3
        order = torch.randperm(pool, device=dev, generator=g).int()  # pages scattered over the pool
        table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=dev)
        for s, a in enumerate(_offsets(need)[:-1]):
            table[s, :need[s]] = order[a:a + need[s]]
        T = sum(new)
        qkv = _normal(g, T, (Hq + 2 * Hkv) * D).to(dt)  # the fused projection's output
        st["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        st["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        st["k_pool"] = _normal(g, pool, Hkv, page, D).to(dt)  # what earlier tokens and sequences left
        st["v_pool"] = _normal(g, pool, Hkv, page, D).to(dt)
        st["cu"], st["lens"], st["table"] = _int32(_offsets(new), dev), _int32(lens, dev), table
        st["wq"] = (1 + 0.2 * _normal(g, D)).to(dt) if case["norm"] else None
        st["wk"] = (1 + 0.2 * _normal(g, D)).to(dt) if case["norm"] else None
        st["positions"] = None  # a token's position is its place in its sequence, unless the caller has others
        if case["far"]:
            start = torch.randint(0, case["far"], (len(lens),), device=dev, generator=g)
            seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), _int32(new, dev).long())
            st["positions"] = (start[seq] + torch.arange(T, device=dev) - st["cu"][seq]).int()
        i = torch.arange(case["R"] // 2, dtype=torch.float64, device=dev)
        st["inv_freq"] = torch.exp(-math.log(case["base"]) * 2 * i / max(1, case["R"]))
    else:
        group, cu, prefix, lens = _batch(case)
        # A prefix's pages, in each sequence's table as far as they are full; a prefix's last, partly filled page is
        # copied into the first page that a sequence has for itself.
        full = [p // page for p in prefix]
        pages = [-(-p // page) for p in prefix]
        kept = [full[k] if k >= 0 else 0 for k in group]
        need = [-(-n // page) - kept[s] for s, n in enumerate(lens)]
        pool = sum(pages) + sum(need) + 3
        order = torch.randperm(pool, device=dev, generator=g).int()
        st["k_pool"] = torch.zeros(pool, Hkv, page, D, dtype=dt, device=dev)
        st["v_pool"] = torch.zeros(pool, Hkv, page, D, dtype=dt, device=dev)
        starts = _offsets(pages)
        tables = [order[a:b] for a, b in zip(starts, starts[1:])]
        table = torch.full((len(lens), max(-(-n // page) for n in lens)), -1, dtype=torch.int32, device=dev)
        a = starts[-1]
        for s, k in enumerate(group):
            if k >= 0:
                table[s, :full[k]] = tables[k][:full[k]]
            table[s, kept[s]:kept[s] + need[s]] = order[a:a + need[s]]
            a += need[s]
        # rows of all prefixes, then of what each sequence has for itself
        for name, make in (("k_pool", _keys), ("v_pool", _normal)):
            x = [make(g, p, Hkv, D).to(dt) for p in prefix]
            for k, rows in enumerate(x):
                t = torch.arange(prefix[k], device=dev)
                st[name][tables[k][t // page].long(), :, t % page] = rows
            for s, k in enumerate(group):
                base = kept[s] * page
                rows = make(g, lens[s] - (prefix[k] if k >= 0 else 0), Hkv, D).to(dt)
                if k >= 0:
                    rows = torch.cat((x[k][base:], rows))
                t = torch.arange(base, lens[s], device=dev)
                st[name][table[s, t // page].long(), :, t % page] = rows
        st["q"] = _normal(g, len(lens), case["rows"], Hq, D).to(dt)
        st["table"], st["lens"] = table, _int32(lens, dev)
        st["prefix_table"] = st["prefix"] = st["groups"] = None
        if case["groups"]:
            wide = torch.full((len(prefix), max(pages)), -1, dtype=torch.int32, device=dev)
            for k, t in enumerate(tables):
                wide[k, :len(t)] = t
            st["prefix_table"], st["prefix"] = wide, _int32(prefix, dev)
            st["groups"] = _int32(cu, dev)
        # what the plain form's shapes need, which a program that schedules batches has on the host
        st["batch"] = (group, cu, prefix, lens)
    if own:
        import gqa_flash_attention_gb300 as sdp
        st["cache"] = sdp.Cache16(st["k_pool"], st["v_pool"])
        if case["op"] == "append":
            st["rope"] = sdp.rope_table(st["inv_freq"], mscale=case["mscale"]) if case["R"] else None
    return st


# ------------------------------------------------------------------ plain forms


def _norm(x, w):
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return y * w.float()


def _rotate(x, cos, sin, R, interleaved):
    """The first R channels of x [T, H, D] turned by the angles of its row, cos and sin [T, 1, R / 2]."""
    rot, rest = x[..., :R], x[..., R:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = rot[..., :R // 2], rot[..., R // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1)


def _plain_append(st):
    c = st["case"]
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    T = st["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(len(n), device=n.device), n, output_size=T)
    place = torch.arange(T, device=n.device) - st["cu"][seq] + st["lens"][seq] - n[seq]
    at = place if st["positions"] is None else st["positions"]
    angle = at.double().unsqueeze(-1) * st["inv_freq"]
    cos, sin = (torch.cos(angle) * c["mscale"]).float().unsqueeze(1), (torch.sin(angle) * c["mscale"]).float().unsqueeze(1)
    q, k = st["q"].float(), st["k"].float()
    if c["norm"]:
        q, k = _norm(q, st["wq"]), _norm(k, st["wk"])
    q, k = _rotate(q, cos, sin, c["R"], c["interleaved"]), _rotate(k, cos, sin, c["R"], c["interleaved"])
    page, off = st["table"][seq, place // c["page"]].long(), place % c["page"]
    st["k_pool"][page, :, off] = k.to(st["k"].dtype)
    st["v_pool"][page, :, off] = st["v"]
    return q.to(st["q"].dtype), st["k_pool"], st["v_pool"]


def _rows_of(pool, table, first, end):
    """Rows of tokens [first, end) through block tables [..., pages] in fp32: [..., tokens, Hkv, D]."""
    t = torch.arange(first, end, device=pool.device)
    return pool[table[..., t // pool.shape[2]].clamp_min(0).long(), :, t % pool.shape[2]].float()


def _plain_shared(st):
    c = st["case"]
    Hkv, G, n = c["Hkv"], c["Hq"] // c["Hkv"], c["rows"]
    group, cu, prefix, lens = st["batch"]
    scale = 1 / math.sqrt(c["D"])
    q = st["q"].float().unflatten(2, (Hkv, G))  # [nseq, rows, Hkv, G, D]
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:-1], device=q.device)
    spans = [(cu[k], cu[k + 1], prefix[k], k) for k in range(len(prefix))] or [(0, len(lens), 0, -1)]
    for a, b, P, k in spans:
        if a == b:
            continue
        # the prefix, its rows once for all sequences; every query row sees all of it
        kp, vp = ((_rows_of(st[x], st["prefix_table"][k], 0, P) for x in ("k_pool", "v_pool")) if P else
                  (q.new_zeros(0, Hkv, c["D"]),) * 2)
        sp = torch.einsum("sngid,kgd->gsnik", q[a:b], kp) * scale
        # what each sequence has for itself, padded to the longest
        end = max(lens[a:b])
        ks, vs = (_rows_of(st[x], st["table"][a:b], P, end) for x in ("k_pool", "v_pool"))
        ss = torch.einsum("sngid,skgd->gsnik", q[a:b], ks) * scale
        j = torch.arange(P, end, device=q.device)
        at = st["lens"][a:b, None] - n + torch.arange(n, device=q.device)  # [nseq, rows]
        ss = ss.masked_fill((j > at.unsqueeze(-1))[None, :, :, None], -math.inf)
        m = ss.amax(-1, keepdim=True)
        if P:
            m = torch.maximum(m, sp.amax(-1, keepdim=True))
        m = torch.where(m.isinf(), torch.zeros_like(m), m)
        ep, es = torch.exp(sp - m), torch.exp(ss - m)
        l = ep.sum(-1) + es.sum(-1)
        x = torch.einsum("gsnik,kgd->gsnid", ep, vp) + torch.einsum("gsnik,skgd->gsnid", es, vs)
        x = x / torch.where(l > 0, l, torch.ones_like(l)).unsqueeze(-1)
        o[a:b] = x.permute(1, 2, 0, 3, 4)
        lse[a:b] = (torch.log(l) + m.squeeze(-1)).permute(1, 2, 0, 3)
    return o.flatten(2, 3).to(st["q"].dtype), lse.flatten(2, 3)


def run(state):
    c = state["case"]
    if not own:
        return _plain_append(state) if c["op"] == "append" else _plain_shared(state)
    import gqa_flash_attention_gb300 as sdp
    if c["op"] == "append":
        q = sdp.cache16_append(state["cache"], state["k"], state["v"], state["cu"], state["lens"], state["table"],
                               rope=state["rope"], q=state["q"], positions=state["positions"], q_weight=state["wq"],
                               k_weight=state["wk"], eps=1e-6, interleaved=c["interleaved"])
        return q, state["cache"].k, state["cache"].v
    return sdp.fwd_cache16(state["q"], state["cache"], state["lens"], state["table"], prefix_table=state["prefix_table"],
                           prefix_lens=state["prefix"], cu_groups=state["groups"])


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    c, D = case, case["D"]
    if c["op"] == "append":
        lens = _lens(c)
        new = sum(_new(c, lens))
        rows = new * (c["Hq"] + c["Hkv"])
        w = 4 * D if c["norm"] else 0
        return {"bytes": 4 * D * (rows + new * c["Hkv"]) + w + 4 * c["R"] + (4 * new if c["far"] else 0) + 12 * len(lens),
                "flops": rows * ((4 * D if c["norm"] else 0) + 3 * c["R"])}
    group, cu, prefix, lens = _batch(c)
    n = c["rows"]
    keys = sum(prefix[k] for k in range(len(prefix)) if cu[k + 1] > cu[k])
    keys += sum(x - (prefix[k] if k >= 0 else 0) for x, k in zip(lens, group))
    pairs = sum(max(0, p + 1) for x in lens for p in range(x - n, x))
    rows = len(lens) * n * c["Hq"]
    return {"bytes": 4 * D * c["Hkv"] * keys + rows * (4 * D + 4) + 4 * len(lens) + 4 * (keys // c["page"]),
            "flops": 4 * D * c["Hq"] * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits


def _turn(x, pos, freq, R, interleaved, mscale):
    """Rows x [n, H, D] (64 bits) at positions pos [n]: channel pairs as complex numbers times exp(i pos f)."""
    ang = pos.double()[:, None] * freq[None]
    z = torch.polar(torch.full_like(ang, mscale), ang)[:, None]
    pairs = x[..., :R].reshape(*x.shape[:-1], R // 2, 2) if interleaved else torch.stack((x[..., :R // 2], x[..., R // 2:R]), -1)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    y = y.flatten(-2) if interleaved else torch.cat((y[..., 0], y[..., 1]), -1)
    return torch.cat((y, x[..., R:]), -1)


def exact(case, seed):
    global own
    was, own = own, False
    st = prepare(case, seed)
    own = was
    c, D = case, case["D"]
    if c["op"] == "append":
        if st["q"].numel() > 1 << 29:
            return None
        cu, lens = st["cu"].tolist(), st["lens"].tolist()
        place = torch.cat([torch.arange(n - (b - a), n, device=st["q"].device) for a, b, n in zip(cu, cu[1:], lens)])
        seq = torch.cat([torch.full((b - a,), s, device=place.device) for s, (a, b) in enumerate(zip(cu, cu[1:]))])
        at = place if st["positions"] is None else st["positions"]
        out = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            y = x.double()
            if c["norm"]:
                y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / D + 1e-6) * w.double()
            if c["R"]:
                y = _turn(y, at, st["inv_freq"], c["R"], c["interleaved"], c["mscale"])
            out.append(y)
        ids = st["table"][seq, torch.div(place, c["page"], rounding_mode="floor")].long()
        pools = [st["k_pool"].double(), st["v_pool"].double()]
        for pool, rows in zip(pools, (out[1], st["v"].double())):
            pool[ids, :, place % c["page"]] = rows
        return (out[0], *pools)
    group, cu, prefix, lens = _batch(c)
    Hkv, G, n = c["Hkv"], c["Hq"] // c["Hkv"], c["rows"]
    os_, ls = [], []
    for s, length in enumerate(lens):
        # the whole sequence through its own table, in which a prefix's full pages stand too
        t = torch.arange(length, device=st["q"].device)
        ids = st["table"][s, t // c["page"]].long()
        k, v = (st[x][ids, :, t % c["page"]].double().transpose(0, 1) for x in ("k_pool", "v_pool"))  # [Hkv, len, D]
        q = st["q"][s].double().view(n, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, n * G, D)
        z = (q @ k.transpose(1, 2)).view(Hkv, n, G, length) / math.sqrt(D)
        seen = t[None] <= (length - n + torch.arange(n, device=t.device))[:, None]
        z = z.masked_fill(~seen[None, :, None], -math.inf)
        l = torch.logsumexp(z, -1)
        w = torch.exp(z - torch.where(l.isinf(), torch.zeros_like(l), l)[..., None])
        o = (w.view(Hkv, n * G, length) @ v).view(Hkv, n, G, D)
        os_.append(o.permute(1, 0, 2, 3).reshape(n, Hkv * G, D))
        ls.append(l.permute(1, 0, 2).reshape(n, Hkv * G))
    return torch.stack(os_), torch.stack(ls)
