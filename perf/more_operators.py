"""Cases of the operators around the cache and the experts: norms and rotation of queries and keys,
attention over the 8-bit cache for trees of drafted tokens and for windows with first tokens that
stay visible, routing with the grouped rows that follow from it, and log probabilities of tokens.
Each in its plain form (elementary torch operations) and through the package's entry points.

A cache page holds 64 tokens.  K codes are [page, head, D / 16, 64, 16]; V codes are
[page, head, D, 64] with token 16 j + 4 g + e of the page at place 16 g + 4 j + e.  A value is
its E4M3 code times 2^(b - 127), b being the byte of its (page, head) in the K or V scales.
"""
import math

import torch

own = False

PAGE = 64
EPS = 1e-6


def listed():
    return [
        # one token of 64 sequences, from the fp32 rows that the projection's GEMM writes: latency
        dict(name="rope_decode", op="rope", rows=64, hq=32, hkv=8, d=128, rot=128, pairs="halves",
             norm=True, dtype="fp32", far=131072),
        # a prompt's BF16 projections
        dict(name="rope_prompt", op="rope", rows=16384, hq=32, hkv=8, d=128, rot=128,
             pairs="halves", norm=True, dtype="bf16", far=32768),
        # one user's tree of drafted tokens: latency
        dict(name="tree_one", op="attend", seqs=1, q=25, kv=1500, hq=32, hkv=8, d=128, window=0,
             sinks=0, tree=True),
        # a batch of trees over ragged contexts
        dict(name="tree_batch", op="attend", seqs=16, q=48, kv=6000, hq=32, hkv=8, d=128,
             window=0, sinks=0, tree=True),
        # a serving batch with long contexts, of which a window and the first tokens are seen
        dict(name="sinks_decode", op="attend", seqs=64, q=1, kv=16384, hq=32, hkv=8, d=128,
             window=4096, sinks=4, tree=False),
        # a chunk of a prompt under the same kind of mask
        dict(name="sinks_chunk", op="attend", seqs=2, q=1024, kv=12000, hq=16, hkv=4, d=128,
             window=2048, sinks=64, tree=False),
        # a decode batch through a router with sigmoid scores, a bias for balance and groups
        dict(name="route_decode", op="route", tokens=64, experts=256, topk=8, score="sigmoid",
             bias=True, groups=8, keep=4, top=2, renorm=True, factor=2.5, dtype="fp32"),
        # a prompt through a softmax router
        dict(name="route_prompt", op="route", tokens=16384, experts=128, topk=8, score="softmax",
             bias=False, groups=1, keep=1, top=1, renorm=True, factor=1.0, dtype="fp32"),
        # the rows of each expert, for the grouped quantizer: the decode batch, and a prompt
        dict(name="group_decode", op="group", tokens=64, experts=256, topk=8, pad=128, holes=0.0),
        dict(name="group_prompt", op="group", tokens=16384, experts=256, topk=8, pad=128,
             holes=0.0),
        # one answer's next token, with alternatives: latency
        dict(name="logprobs_one", op="logprobs", rows=1, vocab=128000, given=1, top=5,
             dtype="fp32"),
        # every token of prompts scored
        dict(name="logprobs_prompt", op="logprobs", rows=2048, vocab=128000, given=1, top=20,
             dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(n, lo), hi)


def draw(rng):
    while True:                                              # no dearer than the listed cases
        c = _drawn(rng)
        w = work(c)
        if w["bytes"] < 5.2e8 and w["flops"] < 4.0e10:
            return c


def _drawn(rng):
    op = rng.choice(["rope", "attend", "attend", "route", "group", "logprobs"])
    if op == "rope":
        d = rng.choice([64, 128, 128, 256, 80, 96])
        hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, rows=_log_int(rng, 1, 16384), hq=hkv * rng.choice([1, 2, 3, 4, 7, 8]),
                    hkv=hkv, d=d, rot=rng.choice([d, d, 16 * rng.randint(1, d // 16)]),
                    pairs=rng.choice(["halves", "neighbours"]), norm=rng.random() < 0.7,
                    dtype=rng.choice(["fp32", "bf16"]), far=_log_int(rng, 100, 1000000))
    if op == "attend":
        hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        tree = rng.random() < 0.6
        if tree:
            q = _log_int(rng, 2, 150)
            kv = q + _log_int(rng, 1, 20000)
        elif rng.random() < 0.6:
            q = rng.choice([1, 1, 2, 5])
            kv = q + _log_int(rng, 1, 50000)
        else:
            q = _log_int(rng, 9, 1024)
            kv = q + rng.randint(0, 8000)
        seqs = _log_int(rng, 1, max(1, min(64, 262144 * 2 // (kv * hkv), 2048 // q)))
        window = rng.choice([0, _log_int(rng, 1, 5000)]) if tree else _log_int(rng, 1, 5000)
        return dict(op=op, seqs=seqs, q=q, kv=kv, hq=hq, hkv=hkv, d=d, window=window,
                    sinks=rng.choice([0, 1, 4, rng.randint(2, 200)]) if window else 0, tree=tree)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * _log_int(rng, 8 if groups == 1 else 4, 512 // groups)
        keep = rng.randint(1, groups) if groups > 1 else 1
        most = min(16, experts // groups * keep)
        return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts,
                    topk=rng.randint(1, most), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.6, factor=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["fp32", "fp32", "bf16"]))
    if op == "group":
        experts = _log_int(rng, 4, 1024)
        return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts,
                    topk=rng.randint(1, min(12, experts)), pad=rng.choice([16, 32, 128]),
                    holes=rng.choice([0.0, 0.3]))
    rows = _log_int(rng, 1, 2000)
    return dict(op=op, rows=rows, vocab=_log_int(rng, 100, min(262144, 250000000 // rows)),
                given=rng.choice([1, 1, 3, 8]), top=rng.choice([0, 1, 5, 20, 32]),
                dtype=rng.choice(["fp32", "bf16"]))


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randint(g, lo, hi, shape):
    """int32 in [lo, hi], both ends included."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _e4m3(g, shape):
    """E4M3 codes of normal values of spread 60 (no NaN code)."""
    x = _randn(g, shape, torch.float16)
    return (x * 60).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _ragged(g, n, least, most):
    """n lengths from `most` down to about `least`, in random order."""
    lens = [most - i * (most - least) // n for i in range(n)]
    order = torch.randperm(n, generator=g, device="cuda")
    return torch.tensor(lens, dtype=torch.int32, device="cuda")[order].contiguous()


def _tree_masks(g, n, most):
    """Masks of random trees, each node's parent being one of the eight nodes before it or the
    root: bit j of a row's words is set where it sees its sequence's row j."""
    S, words = n.numel(), (most + 63) // 64
    back = _randint(g, 1, 8, (S, most))
    masks = torch.zeros((S, most + 1, words), dtype=torch.int64, device="cuda")
    seq = torch.arange(S, device="cuda")
    for i in range(most):                                    # parent `most` is the root
        parent = i - back[:, i].long()
        masks[:, i] = masks[seq, torch.where(parent < 0, most, parent)]
        masks[:, i, i // 64] |= 1 << (i % 64) if i % 64 < 63 else -(1 << 63)
    real = torch.arange(most, device="cuda")[None] < n[:, None]
    return masks[:, :most][real].contiguous()


def _prepare_rope(c, g, s):
    width = (c["hq"] + 2 * c["hkv"]) * c["d"]
    x = _randn(g, (c["rows"], width)) * torch.exp2(_randint(g, -2, 2, (c["rows"], 1)).float())
    x = x.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
    x = x.view(c["rows"], c["hq"] + 2 * c["hkv"], c["d"])
    s["q"], s["k"], s["v"] = x.split([c["hq"], c["hkv"], c["hkv"]], 1)
    s["q_weight"] = s["k_weight"] = None
    if c["norm"]:
        s["q_weight"] = 1 + 0.1 * _randn(g, (c["d"],))
        s["k_weight"] = 1 + 0.1 * _randn(g, (c["d"],))
    i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
    s["inv_freq"] = 10000.0 ** (-2 * i / c["rot"])
    s["positions"] = _randint(g, 0, c["far"], (c["rows"],))


def _prepare_attend(c, g, s):
    most = min(c["q"], c["kv"])
    n = _ragged(g, c["seqs"], max(1, most * 3 // 4), most)
    lens = torch.maximum(n, _ragged(g, c["seqs"], max(1, c["kv"] // 4), c["kv"]))
    used = (lens + PAGE - 1) // PAGE
    width, pages = (c["kv"] + PAGE - 1) // PAGE, int(used.sum()) + 3
    at = (torch.cumsum(used, 0) - used)[:, None] + torch.arange(width, device="cuda")[None]
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    valid = torch.arange(width, device="cuda")[None] < used[:, None]
    s["table"] = torch.where(valid, order[at.clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
    H, d = c["hkv"], c["d"]
    s["k"], s["v"] = _e4m3(g, (pages, H, d // 16, PAGE, 16)), _e4m3(g, (pages, H, d, PAGE))
    s["ks"] = _randint(g, 119, 122, (pages, H)).to(torch.uint8)
    s["vs"] = _randint(g, 119, 122, (pages, H)).to(torch.uint8)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["lens"], s["offsets"] = lens, torch.cat([zero, torch.cumsum(n, 0).to(torch.int32)])
    s["rows"], s["max_n"], s["max_kv"] = int(n.sum()), int(n.max()), int(lens.max())
    s["q"] = _randn(g, (s["rows"], c["hq"], d)).to(torch.bfloat16)
    s["masks"] = _tree_masks(g, n, s["max_n"]) if c["tree"] else None


def prepare(case, seed):
    g, c, op = _gen(seed), dict(case), case["op"]
    s = dict(case=c)
    if op == "rope":
        _prepare_rope(c, g, s)
    elif op == "attend":
        _prepare_attend(c, g, s)
    elif op == "route":
        z = _randn(g, (c["tokens"], c["experts"])) * 1.5
        s["logits"] = z.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        s["bias"] = 0.05 * _randn(g, (c["experts"],)) if c["bias"] else None
    elif op == "group":
        # distinct experts of a token; some experts are asked for more often than others
        liking = 0.7 * _randn(g, (1, c["experts"])) + torch.rand(
            (c["tokens"], c["experts"]), generator=g, device="cuda")
        ids = liking.argsort(1)[:, :c["topk"]].to(torch.int32)
        holes = torch.rand(ids.shape, generator=g, device="cuda") < c["holes"]
        s["ids"] = torch.where(holes, -1, ids).contiguous()
    else:
        z = _randn(g, (c["rows"], c["vocab"])) * 2.5
        s["logits"] = z.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        s["tokens"] = _randint(g, 0, c["vocab"] - 1, (c["rows"], c["given"]))
    return s


# ------------------------------------------------------------------ plain forms


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = c["rot"]

    def turn(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        if c["pairs"] == "halves":
            a, b = x[..., :r // 2], x[..., r // 2:r]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([y, x[..., r:]], -1).to(torch.bfloat16)

    out = {"q": turn(s["q"], s["q_weight"]), "k": turn(s["k"], s["k_weight"])}
    if c["dtype"] == "fp32":                                 # BF16 rows of v are used as they are
        out["v"] = s["v"].to(torch.bfloat16)
    return out


def _f8(codes):
    return codes.view(torch.float8_e4m3fn)


def _exp2_of(byte):
    return torch.exp2(byte.float() - 127.0)


def _bits(words):
    """Set bits of each row's words."""
    b = torch.arange(64, device="cuda")
    return ((words[..., None] >> b) & 1).sum((-1, -2))


def _plain_attend(s):
    c = s["case"]
    hq, hkv, d, W = c["hq"], c["hkv"], c["d"], c["window"]
    G, S, N = hq // hkv, c["seqs"], s["max_n"]
    n = s["offsets"][1:] - s["offsets"][:-1]
    base = (s["lens"] - n).long()                            # tokens before the rows
    i = torch.arange(N, device="cuda")
    row = (s["offsets"][:-1, None] + i[None]).long().clamp(max=s["rows"] - 1)
    real = i[None] < n[:, None]
    width = s["table"].shape[1]
    if W:                                                    # the pages of the sinks, then the window's
        head = (c["sinks"] + PAGE - 1) // PAGE
        first = ((base - W) // PAGE).clamp(min=0)
        page = first[:, None] + torch.arange((W + N) // PAGE + 3, device="cuda")
        page = torch.cat([torch.arange(head, device="cuda").expand(S, head),
                          torch.where(page < head, width, page)], 1)
    else:
        page = torch.arange(width, device="cuda").expand(S, width)
    t = s["table"].gather(1, page.clamp(max=width - 1)).long()
    M = t.shape[1]
    k = _f8(s["k"][t]).float() * _exp2_of(s["ks"][t])[..., None, None, None]
    k = k.permute(0, 2, 1, 4, 3, 5).reshape(S, hkv, M * PAGE, d)
    v = _f8(s["v"][t]).float() * _exp2_of(s["vs"][t])[..., None, None]
    v = v.view(S, M, hkv, d, 4, 4, 4).permute(0, 2, 1, 5, 4, 6, 3).reshape(S, hkv, M * PAGE, d)
    j = (page[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1)[:, None]
    j = torch.where(page[:, :, None].expand(S, M, PAGE).flatten(1)[:, None] < width, j, 1 << 40)
    base, at = base[:, None, None], (base[:, None] + i[None])[..., None]
    if c["tree"]:
        words = s["masks"][row]                              # [S, N, words]
        bit = (j - base).clamp(0, 64 * words.shape[-1] - 1)
        drafted = (words.gather(2, (bit // 64).expand(S, N, -1)) >> (bit % 64)) & 1
        near = j >= base - (W - _bits(words)[..., None]) if W else j >= 0
        seen = ((j < base) & (near | (j < c["sinks"]))
                | (j >= base) & (j < s["lens"][:, None, None]) & (drafted != 0))
    else:
        seen = (j <= at) & ((j > at - W) | (j < c["sinks"]) if W else j >= 0)
    q = s["q"][row].float().view(S, N, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(S, hkv, G * N, d)
    x = torch.matmul(q, k.transpose(2, 3).contiguous()) * (d ** -0.5)
    x = x.view(S, hkv, G, N, M * PAGE).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = (x - top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(S, hkv, G * N, M * PAGE), v).view(S, hkv, G, N, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(S, N, hq, d)[real]
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(S, N, hq)[real]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _plain_route(s):
    c = s["case"]
    T, E = c["tokens"], c["experts"]
    z = s["logits"].double()                                 # 64 bits: choices next to each other
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-z))
    else:
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    choice = p if s["bias"] is None else p + s["bias"].double()
    if c["groups"] > 1:
        best = torch.sort(choice.view(T, c["groups"], -1), dim=2, descending=True)[0]
        score = best[..., :c["top"]].sum(2)
        kept = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :c["keep"]]
        open_ = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
        open_ = open_.repeat_interleave(E // c["groups"], 1)
        choice = torch.where(open_, choice, -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True)[1][:, :c["topk"]]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * c["factor"]).float()}


def _plain_group(s):
    c = s["case"]
    E, k = c["experts"], c["topk"]
    flat = s["ids"].view(-1)
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, E).long()
    order = torch.sort(key, stable=True)[1]
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    counts = counts.scatter_add_(0, key, torch.ones_like(key))[:E]
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    rows = torch.cat([zero, torch.cumsum(counts, 0)])
    padded = torch.cat([zero, torch.cumsum((counts + c["pad"] - 1) // c["pad"] * c["pad"], 0)])
    at = torch.arange(flat.numel(), device="cuda")
    entry = torch.zeros_like(at).scatter_(0, order, at)
    return _group_outputs(rows.to(torch.int32), padded.to(torch.int32),
                          torch.where(at < rows[E], order // k, -1).to(torch.int32),
                          torch.where(valid, entry, -1).view(-1, k).to(torch.int32))


def _group_outputs(rows, padded, indices, entries):
    return {"row_offsets": rows, "scales_offsets": padded, "row_indices": indices,
            "entry_rows": entries}


def _plain_logprobs(s):
    c = s["case"]
    z = s["logits"].float()
    m = z.amax(1, keepdim=True)
    x = z - m
    p = torch.exp(x)
    total = p.sum(1, keepdim=True)
    log_total = torch.log(total)
    out = {"logprobs": z.gather(1, s["tokens"].long()) - m - log_total,
           "entropy": (log_total - (p * x).sum(1, keepdim=True) / total)[:, 0]}
    if c["top"]:
        # as one whole number: the value's order, then the lower id first
        b = (z + 0.0).view(torch.int32).long()
        b = torch.where(b < 0, -(b & 0x7FFFFFFF), b)
        key = (b << 32) | (c["vocab"] - torch.arange(c["vocab"], device="cuda"))
        ids = c["vocab"] - (torch.topk(key, c["top"], dim=1)[0] & 0xFFFFFFFF)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = z.gather(1, ids) - m - log_total
    return out


# ------------------------------------------------------------------ one pass


def run(state):
    s, c, op = state, state["case"], state["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "attend": _plain_attend, "route": _plain_route,
                "group": _plain_group, "logprobs": _plain_logprobs}[op](s)
    import fp8_quantization_amd as bsq
    if op == "rope":
        v = s["v"] if c["dtype"] == "fp32" else None
        q, k, v = bsq.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], v=v,
                                   q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                   interleaved=c["pairs"] == "neighbours")
        return {"q": q, "k": k} if v is None else {"q": q, "k": k, "v": v}
    if op == "attend":
        out, lse = bsq.kv_cache_attention_masked(
            s["q"], bsq.KvCache(s["k"], s["v"], s["ks"], s["vs"]), s["offsets"], s["lens"],
            s["table"], s["max_n"], s["max_kv"], masks=s["masks"], sinks=c["sinks"],
            window=c["window"], return_lse=True)
        return {"out": out, "lse": lse}
    if op == "route":
        ids, weights = bsq.moe_route(s["logits"], c["topk"], score=c["score"], bias=s["bias"],
                                     num_groups=c["groups"], topk_groups=c["keep"],
                                     group_top=c["top"], renormalize=c["renorm"],
                                     factor=c["factor"])
        return {"ids": ids, "weights": weights}
    if op == "group":
        return _group_outputs(*bsq.moe_group_rows(s["ids"], c["experts"], pad=c["pad"]))
    r = bsq.token_logprobs(s["logits"], s["tokens"], top=c["top"])
    out = {"logprobs": r.logprobs, "entropy": r.entropy}
    if c["top"]:
        out.update(top_ids=r.top_ids, top_logprobs=r.top_logprobs)
    return out


# ------------------------------------------------------------------ work and exact values


def work(case):
    c, op = case, case["op"]
    size = 2 if c.get("dtype") == "bf16" else 4
    if op == "rope":
        n = c["rows"] * c["d"] * (c["hq"] + c["hkv"] * (2 if c["dtype"] == "fp32" else 1))
        return {"bytes": n * (size + 2), "flops": 10 * n}
    if op == "attend":
        S, L = c["seqs"], c["kv"]
        mean = (L + (S - 1) * (L + max(1, L // 4)) / 2) / S
        N = min(c["q"], L)
        n = (N + (S - 1) * (N + max(1, N * 3 // 4)) / 2) / S
        pages, seen = mean, max(1.0, mean - n / 2)
        if c["window"]:
            pages = min(mean, c["window"] + n + c["sinks"])
            seen = min(seen, c["window"] + c["sinks"])
        return {"bytes": S * (2 * pages * c["hkv"] * c["d"] + 4 * n * c["hq"] * c["d"]),
                "flops": S * 4 * n * seen * c["hq"] * c["d"]}
    if op == "route":
        return {"bytes": c["tokens"] * (size * c["experts"] + 8 * c["topk"]),
                "flops": 10 * c["tokens"] * c["experts"]}
    if op == "group":
        return {"bytes": c["tokens"] * c["topk"] * 12 + c["experts"] * 8, "flops": 0}
    return {"bytes": c["rows"] * (size * c["vocab"] + 4 + 8 * (c["given"] + c["top"])),
            "flops": 8 * c["rows"] * c["vocab"]}


def _exact_rope(c, s):
    r = c["rot"]
    a = s["positions"].double()[:, None, None] * s["inv_freq"]
    turn = torch.complex(torch.cos(a), torch.sin(a))

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS) * w.double()
        y = x.clone()
        if c["pairs"] == "halves":
            z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
            y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
        else:
            z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * turn
            y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
        return y

    out = {"q": one(s["q"], s["q_weight"]), "k": one(s["k"], s["k_weight"])}
    if c["dtype"] == "fp32":
        out["v"] = s["v"].double()
    return out


def _exact_attend(c, s):
    hq, hkv, d, W = c["hq"], c["hkv"], c["d"], c["window"]
    outs, lses = [], []
    off, lens = s["offsets"].tolist(), s["lens"].tolist()
    place = torch.arange(PAGE, device="cuda")
    place = 16 * (place // 4 % 4) + 4 * (place // 16) + place % 4
    for b in range(c["seqs"]):
        n, L = off[b + 1] - off[b], lens[b]
        base, j = L - n, torch.arange(L, device="cuda")
        seen = torch.zeros((n, L), dtype=torch.bool, device="cuda")
        masks = s["masks"][off[b]:off[b + 1]].tolist() if c["tree"] else [()] * n
        rows = []
        for i in range(n):
            if c["tree"]:
                bits = [x for x in range(n) if masks[i][x // 64] >> (x % 64) & 1]
                rows += [[i, base + x] for x in bits]
                last, left = base, len(bits)
            else:
                last, left = base + i + 1, 0
            seen[i, max(0, last - W + left) if W else 0:last] = True
            seen[i, :min(c["sinks"], last)] = True
        if rows:
            rows = torch.tensor(rows, device="cuda")
            seen[rows[:, 0], rows[:, 1]] = True
        some = torch.nonzero(seen.any(0))[:, 0]              # tokens that any row sees
        seen = seen[:, some]
        pages = s["table"][b, (some // PAGE)].long()
        o = torch.zeros((n, hq, d), dtype=torch.float64, device="cuda")
        z = torch.zeros((n, hq), dtype=torch.float64, device="cuda")
        for h in range(hkv):
            k = _f8(s["k"][pages, h, :, some % PAGE]).double().flatten(1)
            v = _f8(s["v"][pages, h, :, place[some % PAGE]]).double()
            k = k * 2.0 ** (s["ks"][pages, h].double() - 127)[:, None]
            v = v * 2.0 ** (s["vs"][pages, h].double() - 127)[:, None]
            for x in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                y = s["q"][off[b]:off[b + 1], x].double() @ k.t().contiguous() / math.sqrt(d)
                y = y.masked_fill(~seen, -math.inf)
                z[:, x] = torch.logsumexp(y, 1)
                o[:, x] = torch.softmax(y, 1) @ v
        outs.append(o)
        lses.append(z)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_route(c, s):
    """Weights of the experts that each token's scores choose, found by repeated maxima."""
    z = s["logits"].double()
    p = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
    left = p.clone() if s["bias"] is None else p + s["bias"].double()
    T, size = c["tokens"], c["experts"] // c["groups"]
    if c["groups"] > 1:
        g = left.view(T, c["groups"], size)
        score = g.topk(min(c["top"], size), 2)[0].sum(2)
        for _ in range(c["groups"] - c["keep"]):             # the lowest group goes, the last of equals
            worst = c["groups"] - 1 - score.flip(1).argmin(1)
            score[torch.arange(T, device="cuda"), worst] = math.inf
            g[torch.arange(T, device="cuda"), worst] = -math.inf
    w = []
    for _ in range(c["topk"]):
        best = left.argmax(1, keepdim=True)
        w.append(p.gather(1, best))
        left.scatter_(1, best, -math.inf)
    w = torch.cat(w, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": None, "weights": w * c["factor"]}


def _exact_logprobs(c, s):
    logp, entropy, top = [], [], []
    for z, t in zip(s["logits"].split(64), s["tokens"].split(64)):
        y = torch.log_softmax(z.double(), 1)
        logp.append(y.gather(1, t.long()))
        entropy.append(-(y.exp() * y).sum(1))
        if c["top"]:
            top.append(y.topk(c["top"], 1)[0])
    out = {"logprobs": torch.cat(logp), "entropy": torch.cat(entropy)}
    if c["top"]:
        out.update(top_ids=None, top_logprobs=torch.cat(top))
    return out


def exact(case, seed):
    if case["op"] == "group":                                # whole numbers alone
        return None
    s, op = prepare(case, seed), case["op"]
    return {"rope": _exact_rope, "attend": _exact_attend, "route": _exact_route,
            "logprobs": _exact_logprobs}[op](case, s)
