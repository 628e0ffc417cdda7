"""Cases of the serving operators: the 8-bit KV cache (append, attention and
page management) and the mixture-of-experts layer for a few tokens, each in
its plain form (elementary torch operations in 32 bits) and through the
package's entry points.

A cache page holds 64 tokens.  K codes are [page, head, D / 16, 64, 16]; V
codes are [page, head, D, 64] with token 16 j + 4 g + e of the page at place
16 g + 4 j + e.  A value is its E4M3 code times 2^(b - 127), b being the byte
of its (page, head) in the K or V scales.
"""
import math

import torch

own = False

PAGE = 64
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one new token for each of 64 running sequences: latency
        dict(name="append_token", op="append", seqs=64, new=1, old=1000, hkv=8, d=128),
        # prompts of 8 sequences, some of them continued inside a page
        dict(name="append_prompt", op="append", seqs=8, new=2048, old=100, hkv=8, d=128),
        # one user, a short conversation: latency
        dict(name="decode_one", op="attend", seqs=1, q=1, kv=777, hq=32, hkv=8, d=128, window=0),
        # a serving batch of ragged lengths
        dict(name="decode_batch", op="attend", seqs=64, q=1, kv=8192, hq=32, hkv=8, d=128,
             window=0),
        # two long documents: the work is split over the tokens
        dict(name="decode_long", op="attend", seqs=2, q=1, kv=131072, hq=32, hkv=4, d=128,
             window=0),
        # a few proposed tokens verified at once, one head to a head, sliding window
        dict(name="verify_tokens", op="attend", seqs=16, q=5, kv=2500, hq=8, hkv=8, d=64,
             window=1024),
        # a chunk of a prompt over what the cache already holds
        dict(name="prompt_chunk", op="attend", seqs=2, q=2048, kv=8192, hq=32, hkv=8, d=128,
             window=0),
        # 32 samples forked from 32 prompts and freed again
        dict(name="fork_free", op="fork", seqs=32, kv=4000, pages=4096, hkv=4, d=64),
        # a pool half free: its live pages moved together
        dict(name="compact_pool", op="compact", seqs=64, kv=8000, pages=8192, hkv=8, d=128),
        # one token through 128 experts, 8 of them chosen from the router's logits
        dict(name="moe_one_token", op="moe", tokens=1, experts=128, topk=8, h=2048, i=768,
             fmt="mxfp4", logits=True),
        # a decode batch over 256 experts of the width the prefill GEMM is measured at
        dict(name="moe_batch", op="moe", tokens=16, experts=256, topk=8, h=7168, i=512,
             fmt="mxfp4", logits=True),
        # E4M3 weights, the caller's own routing, every expert in use
        dict(name="moe_mxfp8", op="moe", tokens=64, experts=64, topk=4, h=4096, i=1024,
             fmt="mxfp8", logits=False),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(n, lo), hi)


def draw(rng):
    while True:                                              # no dearer than the listed cases
        c = _drawn(rng)
        w = work(c)
        if w["bytes"] < 8.0e8 and w["flops"] < 3.5e11 and 3 * 1024 not in c.values():
            return c


def _drawn(rng):
    op = rng.choice(["append", "attend", "attend", "fork", "compact", "moe", "moe"])
    if op == "append":
        new = _log_int(rng, 1, 2000)
        return dict(op=op, seqs=_log_int(rng, 1, max(1, min(64, 16000 // new))), new=new,
                    old=rng.randint(0, 1000), hkv=rng.choice([1, 2, 4, 8]),
                    d=rng.choice([64, 128, 256]))
    if op == "attend":
        hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        if rng.random() < 0.6:
            kv = _log_int(rng, 1, 100001)
            seqs = _log_int(rng, 1, max(1, min(64, 262144 * 4 // (kv * hkv))))
            q = rng.choice([1, 1, 1, 2, 4, 7])
        else:
            q = _log_int(rng, 9, 2047)
            kv = q + rng.randint(0, 6000)
            seqs = max(1, min(4, 4096 // q))
            hq = min(hq, 32)
        return dict(op=op, seqs=seqs, q=q, kv=kv, hq=hq, hkv=hkv, d=d,
                    window=rng.choice([0, 0, 0, rng.randint(1, 4000)]))
    if op in ("fork", "compact"):
        kv = _log_int(rng, 100, 6000)
        seqs = _log_int(rng, 1, 50)
        pages = seqs * (kv // PAGE + 2) * 2 + rng.randint(1, 999)
        return dict(op=op, seqs=seqs, kv=kv, pages=pages, hkv=rng.choice([1, 2, 4]),
                    d=rng.choice([64, 128]))
    h, i = 128 * _log_int(rng, 4, 56), 128 * rng.randint(2, 8)
    experts = max(4, min(_log_int(rng, 8, 256), 128 * 7168 * 1024 // (h * i) // 2))
    return dict(op="moe", tokens=_log_int(rng, 1, 64), experts=experts,
                topk=rng.choice([1, 2, 4]) if experts < 8 else rng.choice([1, 2, 4, 6, 8]),
                h=h, i=i, fmt=rng.choice(["mxfp4", "mxfp4", "mxfp8"]),
                logits=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randint(g, lo, hi, shape):
    """int32 in [lo, hi], both ends included."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _e4m3(g, shape):
    """E4M3 codes of normal values of spread 60 (no NaN code)."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    return (x * 60).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _pool(g, pages, hkv, d):
    return dict(k=_e4m3(g, (pages, hkv, d // 16, PAGE, 16)), v=_e4m3(g, (pages, hkv, d, PAGE)),
                ks=_randint(g, 119, 122, (pages, hkv)).to(torch.uint8),
                vs=_randint(g, 119, 122, (pages, hkv)).to(torch.uint8))


def _ragged(g, n, least, most):
    """n lengths from `most` down to about `least`, in random order."""
    lens = [most - i * (most - least) // n for i in range(n)]
    order = torch.randperm(n, generator=g, device="cuda")
    return torch.tensor(lens, dtype=torch.int32, device="cuda")[order].contiguous()


def _tables(g, lens, pages, width):
    """Tables that deal the pages of the pool to the sequences in random order."""
    used = (lens + PAGE - 1) // PAGE
    first = torch.cumsum(used, 0) - used
    at = first[:, None] + torch.arange(width, device="cuda", dtype=torch.int32)[None]
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    valid = torch.arange(width, device="cuda")[None] < used[:, None]
    return torch.where(valid, order[at.clamp(max=pages - 1)], 0).to(torch.int32).contiguous(), used


def _offsets(n):
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    return torch.cat([zero, torch.cumsum(n, 0).to(torch.int32)])


def prepare(case, seed):
    g, c, op = _gen(seed), dict(case), case["op"]
    s = dict(case=c)
    if op in ("append", "attend"):
        if op == "append":
            n = _ragged(g, c["seqs"], max(1, c["new"] // 4), c["new"])
            lens = n + _randint(g, c["old"] // 2, c["old"], (c["seqs"],))
            width = (c["old"] + c["new"] + PAGE - 1) // PAGE
            pages = c["seqs"] * width + 3
        else:
            most = min(c["q"], c["kv"])
            n = _ragged(g, c["seqs"], max(1, most * 3 // 4), most)
            lens = torch.maximum(n, _ragged(g, c["seqs"], max(1, c["kv"] // 4), c["kv"]))
            width = (c["kv"] + PAGE - 1) // PAGE
            pages = int(((lens + PAGE - 1) // PAGE).sum()) + 3
        s["table"], _ = _tables(g, lens, pages, width)
        s.update(_pool(g, pages, c["hkv"], c["d"]))
        s["lens"], s["offsets"] = lens, _offsets(n)
        s["rows"], s["max_n"], s["max_kv"] = int(n.sum()), int(n.max()), int(lens.max())
        if op == "append":
            kv = torch.randn((s["rows"], 2, c["hkv"], c["d"]), generator=g, device="cuda")
            kv = (kv * 2.0).to(torch.bfloat16)
            s["new_k"], s["new_v"] = kv[:, 0], kv[:, 1]     # slices of one projection's output
        else:
            s["q"] = torch.randn((s["rows"], c["hq"], c["d"]), generator=g,
                                 device="cuda").to(torch.bfloat16)
    elif op in ("fork", "compact"):
        lens = _ragged(g, c["seqs"], max(1, c["kv"] // 4), c["kv"])
        width = (c["kv"] + PAGE - 1) // PAGE + 1
        table, used = _tables(g, lens, c["pages"], width)
        refs = torch.zeros(c["pages"], dtype=torch.int32, device="cuda")
        valid = torch.arange(width, device="cuda")[None] < used[:, None]
        refs.index_add_(0, table[valid].long(), torch.ones_like(table[valid]))
        s.update(_pool(g, c["pages"], c["hkv"], c["d"]))
        s["refs"] = refs
        if op == "fork":                                    # the second half of the slots is empty
            s["table"] = torch.cat([table, torch.zeros_like(table)])
            s["lens"] = torch.cat([lens, torch.zeros_like(lens)])
            s["parents"] = torch.randperm(c["seqs"], generator=g, device="cuda").to(torch.int32)
            s["children"] = c["seqs"] + torch.randperm(c["seqs"], generator=g,
                                                       device="cuda").to(torch.int32)
        else:
            s["table"], s["lens"] = table, lens
    else:
        E, H, I, T = c["experts"], c["h"], c["i"], c["tokens"]
        for name, n, k in (("w13", 2 * I, H), ("w2", H, I)):
            if c["fmt"] == "mxfp4":
                s[name] = torch.randint(0, 256, (E * n, k // 2), generator=g, device="cuda",
                                        dtype=torch.uint8)
                lo = 127 - 2 - int(math.log2(k) / 2) - 1
            else:
                s[name] = _e4m3(g, (E * n, k))
                lo = 127 - 6 - int(math.log2(k) / 2) - 1
            s[name + "s"] = _randint(g, lo, lo + 2, (E * n // 16, (k + 511) // 512 * 256)).to(
                torch.uint8)
        s["x"] = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        s["logits"] = torch.randn((T, E), generator=g, device="cuda") * 1.5
        if not c["logits"]:                                 # a router of the caller's own
            order = torch.rand((T, E), generator=g, device="cuda").argsort(1)
            s["ids"] = order[:, :c["topk"]].to(torch.int32).contiguous()
            w = torch.rand((T, c["topk"]), generator=g, device="cuda") + 0.1
            s["weights"] = w / w.sum(1, keepdim=True)
    return s


# ------------------------------------------------------------------ plain forms


def _exp2_of(byte):
    return torch.exp2(byte.float() - 127.0)


def _f8(codes):
    return codes.view(torch.float8_e4m3fn)


def _cache_values(s):
    """K and V of every sequence in 32 bits: [seqs, heads, tokens, D]."""
    t = s["table"].long()
    S, M = t.shape
    _, H, C, _, _ = s["k"].shape
    k = _f8(s["k"][t]).float() * _exp2_of(s["ks"][t])[..., None, None, None]
    k = k.permute(0, 2, 1, 4, 3, 5).reshape(S, H, M * PAGE, 16 * C)
    v = _f8(s["v"][t]).float() * _exp2_of(s["vs"][t])[..., None, None]
    v = v.view(S, M, H, 16 * C, 4, 4, 4).permute(0, 2, 1, 5, 4, 6, 3)
    return k, v.reshape(S, H, M * PAGE, 16 * C)


def _plain_attend(s):
    c, q = s["case"], s["q"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    G, S, N = hq // hkv, c["seqs"], s["max_n"]
    k, v = _cache_values(s)
    L = k.shape[2]
    n = s["offsets"][1:] - s["offsets"][:-1]
    i = torch.arange(N, device="cuda")
    row = (s["offsets"][:-1, None] + i[None]).long()
    real = i[None] < n[:, None]
    qp = q[row.clamp(max=s["rows"] - 1)].float()             # [S, N, hq, d]
    qp = qp.view(S, N, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(S, hkv, G * N, d)
    x = torch.matmul(qp, k.transpose(2, 3).contiguous()) * (d ** -0.5)
    at = s["lens"][:, None] - n[:, None] + i[None]           # the query's place: [S, N]
    j = torch.arange(L, device="cuda")
    seen = j[None, None] <= at[..., None]
    if c["window"]:
        seen = seen & (j[None, None] > at[..., None] - c["window"])
    x = x.view(S, hkv, G, N, L).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = (x - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, hkv, G * N, L), v).view(S, hkv, G, N, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + total.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(S, N, hq, d)[real]
    return {"out": o.to(torch.bfloat16),
            "lse": lse.permute(0, 3, 1, 2).reshape(S, N, hq)[real]}


def _v_place(t):
    """Where a page's V holds token t of it."""
    return 16 * (t // 4 % 4) + 4 * (t // 16) + t % 4


def _scale_byte(amax):
    """E8M0 byte of E4M3 codes for this largest magnitude (a normal number or 0)."""
    return torch.floor(torch.log2(amax.double().clamp(min=2.0 ** -130))).clamp(min=-119).int() + 119


def _plain_append(s):
    c = s["case"]
    n = s["offsets"][1:] - s["offsets"][:-1]
    r = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["offsets"][1:].contiguous(), r, right=True)
    pos = (s["lens"][seq] - s["offsets"][1:][seq] + r).long()
    page, tok = s["table"][seq, pos // PAGE].long(), pos % PAGE
    old = s["lens"] - n
    kept = old % PAGE                                        # tokens that stay in the first page
    first = s["table"].gather(1, (old // PAGE).clamp(max=s["table"].shape[1] - 1)[:, None].long())
    first, kept = first[:, 0].long()[kept > 0], kept[kept > 0]
    slot = torch.arange(PAGE, device="cuda")
    for name, x in (("k", s["new_k"]), ("v", s["new_v"])):
        x = x.float()                                        # [rows, H, D]
        codes, scales = s[name], s[name + "s"]
        amax = torch.zeros(scales.shape, device="cuda").index_reduce_(0, page, x.abs().amax(-1),
                                                                      "amax")
        byte = _scale_byte(amax)
        was = scales[first].int()
        byte[first] = torch.maximum(byte[first], was)        # a page only ever grows its scale
        factor = torch.exp2((was - byte[first]).float())
        if name == "k":
            cur = codes[first]
            stay = (slot[None] < kept[:, None])[:, None, None, :, None]
            new = (_f8(cur).float() * factor[..., None, None, None]).to(torch.float8_e4m3fn)
        else:
            cur = codes[first]
            stay = torch.zeros((len(first), PAGE), dtype=torch.bool, device="cuda")
            stay = stay.scatter(1, _v_place(slot)[None].expand_as(stay),
                                slot[None] < kept[:, None])[:, None, None, :]
            new = (_f8(cur).float() * factor[..., None, None]).to(torch.float8_e4m3fn)
        codes[first] = torch.where(stay, new.view(torch.uint8), cur)
        y = x * torch.exp2(127.0 - byte[page].float())[..., None]
        y = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        if name == "k":
            codes.permute(0, 3, 1, 2, 4)[page, tok] = y.view(s["rows"], c["hkv"], -1, 16)
        else:
            codes.permute(0, 3, 1, 2)[page, _v_place(tok)] = y
        scales[page] = byte[page].to(torch.uint8)
    return _append_outputs(s)


def _append_outputs(s):
    return {"k": _f8(s["k"]), "v": _f8(s["v"]), "k_scales": s["ks"], "v_scales": s["vs"]}


def _plain_fork(s):
    table, lens, refs = s["table"], s["lens"], s["refs"]
    pa, ch = s["parents"].long(), s["children"].long()
    width = torch.arange(table.shape[1], device="cuda")
    # fork: full pages are shared, a partly filled last page is copied
    n = lens[pa]
    part = n % PAGE != 0
    free = torch.nonzero(refs == 0)[:, 0]
    rank = torch.cumsum(part.int(), 0)
    good = ~part | (rank <= free.numel())
    n = torch.where(good, n, 0)
    full, part = n // PAGE, part & good
    rows = table[pa]
    table[ch] = torch.where(width[None] < (n[:, None] + PAGE - 1) // PAGE, rows, table[ch])
    shared = rows[width[None] < full[:, None]].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    new, last = free[rank[part].long() - 1], rows[part, full[part].long()].long()
    table[ch[part], full[part].long()] = new.to(torch.int32)
    refs[new] = 1
    for name in ("k", "v", "ks", "vs"):
        s[name][new] = s[name][last]
    lens[ch] = n
    held = lens.clone()
    # free: every page of the children loses one user
    rows, used = table[ch], (lens[ch] + PAGE - 1) // PAGE
    gone = rows[width[None] < used[:, None]].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    lens[ch] = 0
    return _fork_outputs(s, (~good).to(torch.int32), held)


def _fork_outputs(s, status, held):
    return {"status": status, "held": held, "table": s["table"], "lens": s["lens"],
            "refs": s["refs"], "k": _f8(s["k"]), "v": _f8(s["v"]), "k_scales": s["ks"],
            "v_scales": s["vs"]}


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    count = live.sum()
    idx = torch.arange(refs.numel(), device="cuda")
    src, dst = idx[live & (idx >= count)], idx[~live & (idx < count)]
    for name in ("k", "v", "ks", "vs"):
        s[name][dst] = s[name][src]
    remap = idx.clone()
    remap[src] = dst
    used = (s["lens"] + PAGE - 1) // PAGE
    valid = torch.arange(table.shape[1], device="cuda")[None] < used[:, None]
    table = torch.where(valid, remap[table.long()].to(torch.int32), table)
    refs = refs.clone()
    refs[dst] = refs[src]
    refs[src] = 0
    return _compact_outputs(s, table, refs, count.to(torch.int32).view(1))


def _compact_outputs(s, table, refs, count):
    return {"table": table, "refs": refs, "live": count, "k": _f8(s["k"]), "v": _f8(s["v"]),
            "k_scales": s["ks"], "v_scales": s["vs"]}


def _weights(s, name, n, k, experts):
    """Weights of the experts (an index tensor, or None for all) as values [len, n, k]."""
    E = s["case"]["experts"]
    codes = s[name].view(E, n, -1)
    rec = s[name + "s"].view(E, n // 16, -1, 4, 16, 4)       # record: block, row, step
    if experts is not None:
        codes, rec = codes[experts], rec[experts]
    b = rec.permute(0, 1, 4, 2, 5, 3).reshape(codes.shape[0], n, -1)[..., :k // 32]
    if s["case"]["fmt"] == "mxfp4":
        values = torch.tensor(FP4 + tuple(-x for x in FP4), device="cuda")
        w = torch.stack([values[(codes & 15).int()], values[(codes >> 4).int()]], -1)
    else:
        w = _f8(codes).float()
    w = w.view(codes.shape[0], n, k // 32, 32) * _exp2_of(b)[..., None]
    return w.view(codes.shape[0], n, k)


def _routing(s):
    c = s["case"]
    if not c["logits"]:
        return s["ids"], s["weights"]
    x = s["logits"]
    ids = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :c["topk"]]
    top = x.gather(1, ids)
    p = torch.exp(top - top[:, :1])
    return ids.to(torch.int32), p / p.sum(1, keepdim=True)


def _plain_moe(s):
    c = s["case"]
    E, H, I, T, k = c["experts"], c["h"], c["i"], c["tokens"], c["topk"]
    ids, weights = _routing(s)
    x = s["x"].float()
    if T * k <= E:                                           # the chosen experts' weights alone
        e = ids.view(-1).long()
        a = torch.bmm(_weights(s, "w13", 2 * I, H, e),
                      x.repeat_interleave(k, 0)[..., None])[..., 0]
        h = a[:, :I] / (1 + torch.exp(-a[:, :I])) * a[:, I:] * weights.view(-1, 1)
        y = torch.bmm(_weights(s, "w2", H, I, e), h[..., None]).view(T, k, H).sum(1)
    else:                                                    # every expert for every token
        a = torch.matmul(x[None], _weights(s, "w13", 2 * I, H, None).transpose(1, 2).contiguous())
        share = torch.zeros((T, E), device="cuda").scatter_add_(1, ids.long(), weights)
        h = a[..., :I] / (1 + torch.exp(-a[..., :I])) * a[..., I:] * share.t()[..., None]
        y = torch.bmm(h, _weights(s, "w2", H, I, None).transpose(1, 2).contiguous()).sum(0)
    return {"y": y.to(torch.bfloat16), "ids": ids, "weights": weights}


# ------------------------------------------------------------------ one pass


def run(state):
    s, c, op = state, state["case"], state["case"]["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "fork": _plain_fork,
                "compact": _plain_compact, "moe": _plain_moe}[op](s)
    import fp8_quantization_amd as bsq
    if op == "moe":
        y, ids, weights = bsq.moe_few_tokens(
            s["x"], c["fmt"], s["w13"], s["w13s"], s["w2"], s["w2s"], c["experts"],
            topk=c["topk"], router_logits=s["logits"] if c["logits"] else None,
            topk_ids=s.get("ids"), topk_weights=s.get("weights"))
        return {"y": y, "ids": ids, "weights": weights}
    cache = bsq.KvCache(s["k"], s["v"], s["ks"], s["vs"])
    if op == "append":
        bsq.kv_cache_append(cache, s["new_k"], s["new_v"], s["offsets"], s["lens"], s["table"],
                            s["max_n"])
        return _append_outputs(s)
    if op == "attend":
        out, lse = bsq.kv_cache_attention(s["q"], cache, s["offsets"], s["lens"], s["table"],
                                          s["max_n"], s["max_kv"], window=c["window"],
                                          return_lse=True)
        return {"out": out, "lse": lse}
    if op == "fork":
        status = bsq.kv_pages_fork(cache, s["table"], s["lens"], s["refs"], s["parents"],
                                   s["children"])
        held = s["lens"].clone()
        bsq.kv_pages_free(s["table"], s["lens"], s["refs"], s["children"])
        return _fork_outputs(s, status, held)
    return _compact_outputs(s, *bsq.kv_pages_compact(cache, s["table"], s["lens"], s["refs"]))


# ------------------------------------------------------------------ work and exact values


def _expected(lo, hi):
    return (lo + hi) / 2


def work(case):
    c, op = case, case["op"]
    if op == "append":
        n = c["new"] + (c["seqs"] - 1) * _expected(max(1, c["new"] // 4), c["new"])
        return {"bytes": n * c["hkv"] * c["d"] * 2 * 3, "flops": n * c["hkv"] * c["d"] * 4}
    if op == "attend":
        S, N, L = c["seqs"], c["q"], c["kv"]
        span = L if not c["window"] else min(L, c["window"] + N)
        mean = (span + (S - 1) * _expected(max(1, span // 4), span)) / S
        n = (N + (S - 1) * _expected(max(1, N * 3 // 4), N)) / S
        seen = mean - (0 if c["window"] else n / 2)
        if c["window"]:
            seen = min(seen, c["window"])
        return {"bytes": S * (2 * mean * c["hkv"] * c["d"] + 4 * n * c["hq"] * c["d"]),
                "flops": S * 4 * n * max(1.0, seen) * c["hq"] * c["d"]}
    if op in ("fork", "compact"):
        page = 2 * PAGE * c["hkv"] * c["d"]
        used = c["seqs"] * (c["kv"] + (c["seqs"] - 1) * _expected(c["kv"] // 4, c["kv"])) / (
            c["seqs"] * PAGE)
        if op == "fork":
            return {"bytes": c["seqs"] * 2 * page + 16 * used + 4 * c["pages"], "flops": 0}
        used = min(used, c["pages"])
        return {"bytes": 2 * page * used * (1 - used / c["pages"]) + 8 * c["pages"] + 8 * used,
                "flops": 0}
    E, H, I, T, k = c["experts"], c["h"], c["i"], c["tokens"], c["topk"]
    active = E * (1 - (1 - k / E) ** T)
    per = 17 / 32 if c["fmt"] == "mxfp4" else 33 / 32
    return {"bytes": active * 3 * H * I * per + T * H * 4, "flops": 6.0 * T * k * H * I}


def _e4m3_exact(x):
    """The nearest E4M3 value of each number (ties to even), at most 448, in 64 bits."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -40))).clamp(min=-6)
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -6), e - 1, e).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(a / step) * step).clamp(max=448) * torch.sign(x)


def _exact_attend(c, s):
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    G, outs, lses = hq // hkv, [], []
    off, lens = s["offsets"].tolist(), s["lens"].tolist()
    t = torch.arange(PAGE, device="cuda")
    for b in range(c["seqs"]):
        n, L = off[b + 1] - off[b], lens[b]
        pages = s["table"][b, :(L + PAGE - 1) // PAGE].long()
        at = torch.arange(L - n, L, device="cuda")
        j = torch.arange(L, device="cuda")
        seen = j[None] <= at[:, None]
        if c["window"]:
            seen &= j[None] > at[:, None] - c["window"]
        o = torch.zeros((n, hq, d), dtype=torch.float64, device="cuda")
        z = torch.zeros((n, hq), dtype=torch.float64, device="cuda")
        for h in range(hkv):
            ks = 2.0 ** (s["ks"][pages, h].double() - 127)
            vs = 2.0 ** (s["vs"][pages, h].double() - 127)
            k = _f8(s["k"][pages, h]).double() * ks[:, None, None, None]   # page, piece, token, 16
            k = k.transpose(1, 2).reshape(-1, d)[:L]
            v = _f8(s["v"][pages, h]).double()[:, :, _v_place(t)] * vs[:, None, None]
            v = v.transpose(1, 2).reshape(-1, d)[:L]
            for g in range(G):
                x = s["q"][off[b]:off[b + 1], h * G + g].double() @ k.t() / math.sqrt(d)
                x = x.masked_fill(~seen, -math.inf)
                z[:, h * G + g] = torch.logsumexp(x, 1)
                o[:, h * G + g] = torch.softmax(x, 1) @ v
        outs.append(o)
        lses.append(z)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_append(c, s):
    off, lens = s["offsets"].tolist(), s["lens"].tolist()
    k, v = _f8(s["k"]).double(), _f8(s["v"]).double()
    for b in range(c["seqs"]):
        n, L = off[b + 1] - off[b], lens[b]
        for p in range((L - n) // PAGE, (L + PAGE - 1) // PAGE):
            page = int(s["table"][b, p])
            lo, hi = max(L - n, p * PAGE), min(L, p * PAGE + PAGE)
            rows = slice(off[b] + lo - (L - n), off[b] + hi - (L - n))
            t0, t1 = lo - p * PAGE, hi - p * PAGE
            place = _v_place(torch.arange(PAGE, device="cuda"))
            for name, pool, x in (("ks", k, s["new_k"]), ("vs", v, s["new_v"])):
                x = x[rows].double()                         # [tokens, heads, D]
                X = torch.floor(torch.log2(x.abs().amax((0, 2)))) - 8
                X = X.clamp(min=-127)
                if t0 > 0:
                    was = s[name][page].double() - 127
                    X = torch.maximum(X, was)
                    f = 2.0 ** (was - X)
                    if name == "ks":
                        pool[page, :, :, :t0] = _e4m3_exact(pool[page, :, :, :t0]
                                                            * f[:, None, None, None])
                    else:
                        pool[page][:, :, place[:t0]] = _e4m3_exact(
                            pool[page][:, :, place[:t0]] * f[:, None, None])
                y = _e4m3_exact(x * 2.0 ** -X[None, :, None])
                if name == "ks":
                    pool[page, :, :, t0:t1] = y.view(hi - lo, c["hkv"], -1, 16).permute(1, 2, 0, 3)
                else:
                    pool[page][:, :, place[t0:t1]] = y.permute(1, 2, 0)
    return {"k": k, "v": v, "k_scales": None, "v_scales": None}


def _exact_fork(c, s):
    refs, lens = s["refs"].tolist(), s["lens"].tolist()
    k, v = _f8(s["k"]).double(), _f8(s["v"]).double()
    free = [p for p, r in enumerate(refs) if r == 0]
    for pa in s["parents"].tolist():
        if lens[pa] % PAGE and free:
            new, last = free.pop(0), int(s["table"][pa, lens[pa] // PAGE])
            k[new], v[new] = k[last], v[last]
    return {"status": None, "held": None, "table": None, "lens": None, "refs": None, "k": k,
            "v": v, "k_scales": None, "v_scales": None}


def _exact_compact(c, s):
    refs = s["refs"].tolist()
    k, v = _f8(s["k"]).double(), _f8(s["v"]).double()
    live = sum(r > 0 for r in refs)
    src = [p for p in range(live, len(refs)) if refs[p] > 0]
    dst = [p for p in range(live) if refs[p] == 0]
    if src:
        k[dst], v[dst] = k[src], v[src]
    return {"table": None, "refs": None, "live": None, "k": k, "v": v, "k_scales": None,
            "v_scales": None}


def _exact_weights(s, name, n, k, e):
    """Weights of expert e in 64 bits, from the definition of codes and scale records."""
    codes = s[name][e * n:(e + 1) * n]
    if s["case"]["fmt"] == "mxfp4":
        b = torch.zeros((n, k), dtype=torch.int64, device="cuda")
        b[:, 0::2], b[:, 1::2] = codes % 16, codes // 16
        exp, frac = b // 2 % 4, (b % 2).double()
        w = torch.where(exp == 0, frac / 2, (1 + frac / 2) * 2.0 ** (exp.double() - 1))
        w = torch.where(b >= 8, -w, w)
    else:
        w = _f8(codes).double()
    r = torch.arange(n, device="cuda")[:, None]
    kb = torch.arange(k, device="cuda")[None] // 32
    at = kb // 16 * 256 + 4 * (r % 16 + 16 * (kb % 4)) + kb % 16 // 4
    return w * 2.0 ** (s[name + "s"][(e * n + r) // 16, at].double() - 127)


def _exact_moe(c, s):
    H, I, T = c["h"], c["i"], c["tokens"]
    if c["logits"]:
        x = s["logits"].double()
        ids = torch.tensor([sorted(range(c["experts"]), key=lambda e, r=r: (-r[e], e))[:c["topk"]]
                            for r in x.tolist()], device="cuda")
        top = x.gather(1, ids)
        w = torch.softmax(top, 1)
    else:
        ids, w = s["ids"].long(), s["weights"].double()
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in sorted(set(ids.flatten().tolist())):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        a = s["x"][t].double() @ _exact_weights(s, "w13", 2 * I, H, e).t()
        h = torch.sigmoid(a[:, :I]) * a[:, :I] * a[:, I:]
        y.index_add_(0, t, (h @ _exact_weights(s, "w2", H, I, e).t())
                     * w[t, j][:, None])
    return {"y": y, "ids": None, "weights": w}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    return {"append": _exact_append, "attend": _exact_attend, "fork": _exact_fork,
            "compact": _exact_compact, "moe": _exact_moe}[op](case, s)
