"""Plain 64-bit forms of the operators of bsq_decoder.h, for their tests, on the CPU, and the
error bounds that the kernels' roundings add up to."""
import numpy as np

U = 2.0 ** -24                                   # half a step of fp32, relative
BF16 = 2.0 ** -8


# ------------------------------------------------------------------ norm and rotation


def norm_rope(x, weight, eps, positions, inv_freq, interleaved):
    """(out, bound) of one of q and k: x [rows, heads, D] float64.

    A head's squares are summed by 8 fused steps a lane and 5 sums over lanes, scaled, offset
    and put through a reciprocal root of one step (2 U): the factor is off by (13 + 2) U / 2 + 2 U,
    and two products follow: 12 U of y.  Cosine and sine in 32 bits: the reduced angle (at most
    0.8) and four or five roundings of numbers up to 1, 4 U; the angle itself, in 64 bits, by
    2^-51 of it.  Products and their sum: 2 U.  Then half a step of BF16."""
    rows, heads, D = x.shape
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    n = len(inv_freq)
    angle = positions.astype(np.float64)[:, None] * inv_freq[None]
    cos, sin = np.cos(angle)[:, None], np.sin(angle)[:, None]
    p = np.arange(n) * 2 if interleaved else np.arange(n)
    r = p + 1 if interleaved else p + n
    out, size = y.copy(), np.abs(y) * 12 * U
    out[..., p] = y[..., p] * cos - y[..., r] * sin
    out[..., r] = y[..., r] * cos + y[..., p] * sin
    both = (np.abs(y[..., p]) + np.abs(y[..., r])) * (18 * U + np.abs(angle)[:, None] * 2.0 ** -50)
    size[..., p] = size[..., r] = both
    return out, np.abs(out) * BF16 + size * (1 + BF16) + 2.0 ** -133


# ------------------------------------------------------------------ attention under masks


def seen_tokens(L, n, i, window, sinks, mask):
    """The tokens that row i of n rows and L tokens sees; mask: the rows it sees, or None."""
    base, j = L - n, np.arange(max(L, 0))
    if mask is None:
        near = (j > base + i - window) | (j < sinks) if window else j >= 0
        return near & (j <= base + i)
    near = (j >= base - (window - len(mask))) | (j < sinks) if window else j >= 0
    return near & (j < base) | np.isin(j, base + np.array(sorted(mask), int))


def attention(cache, q, offsets, lens, table, scale, window=0, sinks=0, masks=None):
    """kv_cache_attention_masked with serving_ref.attention's outputs and bounds, whose terms it
    shares; masks: for each row a set of the rows of its sequence that it sees."""
    rows, hq, D = q.shape
    heads = cache.ks.shape[1]
    out, lse = np.zeros((rows, hq, D)), np.full((rows, hq), -np.inf)
    bo, bl = np.zeros((rows, hq, D)), np.zeros((rows, hq))
    owned = np.zeros(rows, bool)
    for s, L in enumerate(lens):
        lo, hi = int(offsets[s]), int(offsets[s + 1])
        n = hi - lo
        owned[lo:hi] = True
        there = np.zeros(max(L, 0), bool)
        for p in range((L + 63) // 64):
            page = int(table[s][p]) if p < len(table[s]) else -1
            there[64 * p:64 * p + 64] = 0 <= page < cache.ks.shape[0]
        see = [seen_tokens(L, n, i, window, sinks, None if masks is None else
                           {x for x in masks[lo + i] if x < n}) & there for i in range(n)]
        some = np.any(see, 0) if n else there & False
        for h in range(heads):
            k, v = np.zeros((max(L, 0), D)), np.zeros((max(L, 0), D))
            for p in np.unique(np.nonzero(some)[0] // 64):
                m = min(64, L - 64 * p)
                k[64 * p:64 * p + m] = cache.values("k", int(table[s][p]), h, m)
                v[64 * p:64 * p + m] = cache.values("v", int(table[s][p]), h, m)
            for i in range(n):
                if not see[i].any():
                    continue
                K, V = k[see[i]], v[see[i]]
                for col in range(h * (hq // heads), (h + 1) * (hq // heads)):
                    x = q[lo + i, col]
                    z = scale * (K @ x)
                    bad = np.isnan(z).any() or np.isnan(V).any()
                    if bad:
                        out[lo + i, col] = lse[lo + i, col] = np.nan
                        continue
                    m = z.max()
                    w = np.exp(z - m)
                    l = w.sum()
                    out[lo + i, col], lse[lo + i, col] = w @ V / l, m + np.log(l)
                    ds = abs(scale) * (D + 4) * U * (np.abs(K) @ np.abs(x)).max() + \
                        (np.abs(z).max() + 16) * 2.0 ** -22 + 2.0 ** -21
                    cnt = (len(K) + 64) * U
                    tiny = 2.0 ** -36 * np.abs(V).sum(0) / l
                    bo[lo + i, col] = np.abs(out[lo + i, col]) * BF16 + tiny + 2.0 ** -133 + \
                        w @ np.abs(V) / l * (2.0 ** -11 + 2 * ds + 2 * cnt) * (1 + 2.0 ** -7)
                    bl[lo + i, col] = ds + cnt + abs(lse[lo + i, col]) * 2.0 ** -22 + 2.0 ** -20
    return out, lse, bo, bl, owned


def words(masks, n):
    """Sets as int64 [rows, n] words of 64 bits."""
    w = np.zeros((len(masks), n), np.uint64)
    for r, m in enumerate(masks):
        for x in m:
            if x < 64 * n:
                w[r, x // 64] |= np.uint64(1 << (x % 64))
    return w.view(np.int64)


def random_tree(rng, n, most_back=6):
    """For each node the set of its ancestors and itself."""
    masks = []
    for i in range(n):
        parent = i - int(rng.integers(1, most_back + 1))
        masks.append((masks[parent] if parent >= 0 else set()) | {i})
    return masks


# ------------------------------------------------------------------ routing


def route(logits, topk, score, bias=None, groups=1, keep=1, top=1, renormalize=True, factor=1.0):
    """(ids, weights, bound of the weights) of moe_route on float64 logits [tokens, experts].

    An exponential of v (the hardware's base-2 one, its argument rounded) is off by (|v| + 2) 2 U,
    relative; sums add their terms' errors and U for each of up to 22 additions; a quotient, a
    product and 1 + t follow, 6 U; what falls below the smallest normal number may be lost."""
    T, E = logits.shape
    ids, weights, bound = np.zeros((T, topk), int), np.zeros((T, topk)), np.zeros((T, topk))
    b = np.zeros(E) if bias is None else np.where(np.isnan(bias), -np.inf, bias)
    size = E // groups
    for t in range(T):
        z = np.where(np.isnan(logits[t]), -np.inf, logits[t])
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-z))
            else:
                s = np.where(z == z.max(), 1.0, np.exp(z - z.max())) * (z > -np.inf)
                s = s / s.sum() if s.sum() else s
        c = np.where((z == -np.inf) | (b == -np.inf), -np.inf, s + b)
        # without a bias c goes by z, of which the scores may lose the difference
        order = z if bias is None else c
        if groups > 1:
            def of(g):
                best = sorted(c[g * size:(g + 1) * size])[::-1][:min(top, size)]
                if bias is None and len(best) == 1:
                    return order[g * size:(g + 1) * size].max()
                return -np.inf if -np.inf in best else sum(best)
            kept = sorted(range(groups), key=lambda g: (-of(g), g))[:keep]
            open_ = [e for e in range(E) if e // size in kept]
        else:
            open_ = list(range(E))
        ids[t] = sorted(open_, key=lambda e: (-order[e], e))[:topk]
        y = np.where(c[ids[t]] == -np.inf, -np.inf, z[ids[t]])
        if score == "sigmoid":
            m = min(y.max(), 0.0) if renormalize and y.max() > -np.inf else 0.0
            v = np.where(y > 0, -y, y - m)
            with np.errstate(over="ignore", invalid="ignore"):
                w = np.where(y == -np.inf, 0.0, np.exp(np.minimum(y, 0) - m) / (1 + np.exp(-np.abs(y))))
            v, den, far = np.where(y == -np.inf, 0, np.abs(np.minimum(y, 0) - m) + np.minimum(np.abs(y), 90)), 1.0, 0.0
            if renormalize:
                den = w.sum()
                far = (w * (v + 2)).sum() / den if den else 0.0
        else:
            pool = y if renormalize else z
            m = pool.max()
            with np.errstate(invalid="ignore"):
                w = np.where(y == m, 1.0, np.exp(y - m)) * (y > -np.inf)
                all_ = np.where(pool == m, 1.0, np.exp(pool - m)) * (pool > -np.inf)
                v = np.where(w > 0, np.where(y == m, 0.0, m - y), 0.0)
                va = np.where(all_ > 0, np.where(pool == m, 0.0, m - pool), 0.0)
            den = all_.sum()
            far = (all_ * (va + 2)).sum() / den if den else 0.0
        weights[t] = factor * w / den if den else 0.0
        bound[t] = np.abs(weights[t]) * ((v + 2 + far) * 2 + 28) * U + abs(factor) * 2.0 ** -125
    return ids, weights, bound


def group_rows(ids, experts, pad):
    """moe_group_rows with loops."""
    T, k = ids.shape
    groups = [[] for _ in range(experts)]
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < experts:
                groups[ids[t, j]].append((t, j))
    rows, scales = [0], [0]
    index, entry = np.full(T * k, -1), np.full((T, k), -1)
    for g in groups:
        for i, (t, j) in enumerate(g):
            index[rows[-1] + i], entry[t, j] = t, rows[-1] + i
        rows.append(rows[-1] + len(g))
        scales.append(scales[-1] + (len(g) + pad - 1) // pad * pad)
    return np.array(rows), np.array(scales), index, entry


# ------------------------------------------------------------------ log probabilities


def logprobs(logits, tokens, top):
    """(logprobs, entropy, top_ids, top_logprobs, and the bounds of the first, second and fourth) of
    token_logprobs on float64 logits [rows, vocab] and tokens [rows, n].

    With d = z - max, exact but for a rounding: an exponential is off by (|d| + 2) 2 U, relative,
    and a slice's sums come to the row's by another factor of the kind; a sum of up to 32 terms a
    thread, 6 + 2 over the threads and 6 over slices adds 46 U.  The base-2 logarithm of the
    hardware, off by 2 U of it and U, its factor and the difference follow."""
    R, V = logits.shape
    z = np.where(np.isnan(logits), -np.inf, logits)
    out = np.full(tokens.shape, -np.inf)
    entropy, be = np.zeros(R), np.zeros(R)
    ids = np.zeros((R, top), int)
    best, bo, bb = np.full((R, top), -np.inf), np.zeros(tokens.shape), np.zeros((R, top))
    for r in range(R):
        ids[r] = np.lexsort((np.arange(V), -z[r]))[:top] if top else []
        m = z[r].max()
        if m == -np.inf:
            continue
        with np.errstate(invalid="ignore"):
            d = np.where(z[r] == m, 0.0, z[r] - m)
        p = np.exp(d)
        l = p.sum()
        p, dd = p / l, np.where(np.isfinite(d), d, 0.0)
        off_l = (p * (np.abs(dd) + 2)).sum() * 4 * U + 46 * U
        off_log = off_l + 6 * U * np.log(l) + 2 * U

        def one(t):
            y = d[t] - np.log(l)
            return y, (off_log + (abs(d[t]) + abs(y)) * 2 * U + 2.0 ** -126 if np.isfinite(y) else 0.0)
        for j, t in enumerate(tokens[r]):
            if 0 <= t < V:
                out[r, j], bo[r, j] = one(t)
        for j, t in enumerate(ids[r]):
            best[r, j], bb[r, j] = one(t)
        entropy[r] = np.log(l) - (p * dd).sum()
        be[r] = off_log + (p * np.abs(dd) * (4 * np.abs(dd) + 60)).sum() * U + \
            (p * np.abs(dd)).sum() * off_l + 4 * U * (abs(entropy[r]) + np.log(l))
    return out, entropy, ids, best, bo, be, bb
