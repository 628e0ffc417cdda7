"""Plain 64-bit forms of the serving operators, for their tests: the cache's
layout and arithmetic, attention, page management and the mixture-of-experts
layer, with loops and elementary operations on the CPU, and the error bounds
that the kernels' roundings add up to."""
import numpy as np
import torch

PAGE = 64
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e4m3_table():
    """Values of the 256 E4M3 (FN) codes."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if (b & 127) == 127:
            x = np.nan
        v[b] = -x if b & 128 else x
    return v


E4M3 = e4m3_table()
_GRID = E4M3[:127]                    # the nonnegative finite values, ascending


def to_e4m3(x):
    """Codes of the nearest E4M3 values (ties to the even code, saturating), sign kept."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_GRID, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    down, up = a - _GRID[lo], _GRID[hi] - a
    code = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def v_place(t):
    """The place of token t (0 .. 63) in a page's rows of V."""
    t = np.asarray(t)
    return 16 * (t // 4 % 4) + 4 * (t // 16) + t % 4


class Cache:
    """The cache in its own layout, numpy uint8."""

    def __init__(self, pages, heads, dim, fill=0):
        self.k = np.full((pages, heads, dim // 16, PAGE, 16), fill, np.uint8)
        self.v = np.full((pages, heads, dim, PAGE), fill, np.uint8)
        self.ks = np.full((pages, heads), fill, np.uint8)
        self.vs = np.full((pages, heads), fill, np.uint8)

    def arrays(self):
        return self.k, self.v, self.ks, self.vs

    def codes(self, name, page, head, t):
        """Codes of token t of (page, head): [D], as a copy."""
        if name == "k":
            return self.k[page, head, :, t, :].reshape(-1)
        return self.v[page, head, :, v_place(t)].reshape(-1)

    def set_codes(self, name, page, head, t, codes):
        if name == "k":
            self.k[page, head, :, t, :] = codes.reshape(-1, 16)
        else:
            self.v[page, head, :, v_place(t)] = codes

    def scale(self, name):
        return self.ks if name == "k" else self.vs

    def values(self, name, page, head, n):
        """Values of the first n tokens: [n, D]; NaN where the scale is."""
        b = int(self.scale(name)[page, head])
        if name == "k":
            c = self.k[page, head].transpose(1, 0, 2).reshape(PAGE, -1)[:n]
        else:
            c = self.v[page, head][:, v_place(np.arange(n))].T
        if b == 255:
            return np.full(c.shape, np.nan)
        return E4M3[c] * 2.0 ** (b - 127)


def scale_byte(x):
    """E8M0 byte of max(floor(log2 amax) - 8, -127); 255 for a NaN or Inf."""
    a = np.abs(x)
    if not np.all(np.isfinite(a)):
        return 255
    m = a.max(initial=0.0)
    if m == 0:
        return 0
    return max(int(np.frexp(m)[1]) - 1 - 8, -127) + 127


def append(cache, k, v, offsets, lens, table):
    """kv_cache_append on float64 k, v [rows, heads, D]."""
    pages = cache.ks.shape[0]
    for s, L in enumerate(lens):
        lo, hi = int(offsets[s]), int(offsets[s + 1])
        n = hi - lo
        if n <= 0 or L - n < 0:
            continue
        for p in range((L - n) // PAGE, (L + PAGE - 1) // PAGE):
            page = int(table[s][p]) if p < len(table[s]) else -1
            if not 0 <= page < pages:
                continue
            t0, t1 = max(0, L - n - p * PAGE), min(PAGE, L - p * PAGE)
            r0 = lo + p * PAGE + t0 - (L - n)
            for name, x in (("k", k), ("v", v)):
                for h in range(x.shape[1]):
                    new = x[r0:r0 + t1 - t0, h]
                    was = int(cache.scale(name)[page, h]) if t0 > 0 else 0
                    b = scale_byte(new)
                    b = 255 if was == 255 or b == 255 else max(b, was)
                    cache.scale(name)[page, h] = b
                    if b != was:
                        for t in range(t0):
                            c = cache.codes(name, page, h, t)
                            c = c * 0 if b == 255 else to_e4m3(E4M3[c] * 2.0 ** (was - b))
                            cache.set_codes(name, page, h, t, c)
                    for t in range(t0, t1):
                        c = to_e4m3(new[t - t0] * 2.0 ** (127 - b)) if b != 255 else \
                            np.zeros(x.shape[2], np.uint8)
                        cache.set_codes(name, page, h, t, c)


def attention(cache, q, offsets, lens, table, scale, window=0):
    """(out, lse, bound of out, bound of lse) of kv_cache_attention; rows that no sequence
    owns are None-filled with NaN in a mask `owned`.

    Bounds: K, V and q enter exactly.  A score is a sum of D exact products in fp32, scaled
    and offset: off by at most ds.  A weight is off by a factor e^ds, 2^-21 of the exponential
    and, where it meets V, half a step of FP16 (2^-11); sums over n tokens by n 2^-24.  The
    result is rounded to BF16 (2^-8)."""
    rows, hq, D = q.shape
    heads = cache.ks.shape[1]
    out, lse = np.zeros((rows, hq, D)), np.full((rows, hq), -np.inf)
    bo, bl = np.zeros((rows, hq, D)), np.zeros((rows, hq))
    owned = np.zeros(rows, bool)
    for s, L in enumerate(lens):
        lo, hi = int(offsets[s]), int(offsets[s + 1])
        n = hi - lo
        owned[lo:hi] = True
        for h in range(heads):
            K, V, at = [np.zeros((0, D))], [np.zeros((0, D))], [np.zeros(0, int)]
            for p in range((L + PAGE - 1) // PAGE):
                page = int(table[s][p]) if p < len(table[s]) else -1
                if not 0 <= page < cache.ks.shape[0]:
                    continue
                m = min(PAGE, L - p * PAGE)
                K.append(cache.values("k", page, h, m))
                V.append(cache.values("v", page, h, m))
                at.append(p * PAGE + np.arange(m))
            K, V, at = np.concatenate(K), np.concatenate(V), np.concatenate(at)
            for i in range(n):
                P = L - n + i
                see = (at <= P) & ((at > P - window) if window else True)
                if not see.any():
                    continue
                k, v = K[see], V[see]
                for g in range(hq // heads):
                    x = q[lo + i, h * (hq // heads) + g]
                    z = scale * (k @ x)
                    m = np.nanmax(z) if not np.all(np.isnan(z)) else 0.0
                    w = np.exp(z - m)
                    # a NaN scale of either makes NaN of the whole row
                    bad = np.isnan(z).any() or np.isnan(v).any()
                    l = np.nan if bad else w.sum()
                    col = h * (hq // heads) + g
                    out[lo + i, col] = np.nan if bad else w @ v / l
                    lse[lo + i, col] = np.nan if bad else m + np.log(l)
                    if bad:
                        continue
                    ds = abs(scale) * (D + 4) * 2.0 ** -24 * (np.abs(k) @ np.abs(x)).max() + \
                        (np.abs(z).max() + 16) * 2.0 ** -22 + 2.0 ** -21
                    cnt = (len(k) + 64) * 2.0 ** -24
                    spread = w @ np.abs(v) / l
                    # weights below 2^-25 of the largest: an absolute 2^-36 of it each
                    tiny = 2.0 ** -36 * np.abs(v).sum(0) / l
                    bo[lo + i, col] = np.abs(out[lo + i, col]) * 2.0 ** -8 + \
                        spread * (2.0 ** -11 + 2 * ds + 2 * cnt) * (1 + 2.0 ** -7) + tiny + 2.0 ** -133
                    bl[lo + i, col] = ds + cnt + abs(lse[lo + i, col]) * 2.0 ** -22 + 2.0 ** -20
    return out, lse, bo, bl, owned


# ------------------------------------------------------------------ pages


def pages_of(n):
    return (n + PAGE - 1) // PAGE


class Pool:
    """Table, lengths and counts as lists, changed as the kv_pages_* calls state."""

    def __init__(self, table, lens, refs):
        self.table = [list(r) for r in table]
        self.lens, self.refs = list(lens), list(refs)

    def _give(self, needs):
        """Pages for the requests' needs in order; None for one that gets none."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        out, at = [], 0
        for n in needs:
            out.append(free[at:at + n] if n == 0 or at + n <= len(free) else None)
            at += n
        return out

    def reserve(self, slots, add):
        M, needs, status = len(self.table[0]), [], []
        for s, a in zip(slots, add):
            bad = 2 if not 0 <= s < len(self.lens) else \
                1 if a < 0 or self.lens[s] + a > M * PAGE else 0
            status.append(bad)
            needs.append(0 if bad else pages_of(self.lens[s] + a) - pages_of(self.lens[s]))
        for i, got in enumerate(self._give(needs)):
            if status[i]:
                continue
            if got is None:
                status[i] = 1
                continue
            s = slots[i]
            for j, p in enumerate(got):
                self.table[s][pages_of(self.lens[s]) + j] = p
                self.refs[p] = 1
            self.lens[s] += add[i]
        return status

    def fork(self, parents, children, cache=None):
        S, status, needs = len(self.lens), [], []
        for p, c in zip(parents, children):
            bad = 0 if 0 <= p < S and 0 <= c < S else 2
            status.append(bad)
            needs.append(0 if bad else int(self.lens[p] % PAGE != 0))
        for i, got in enumerate(self._give(needs)):
            p, c = parents[i], children[i]
            if status[i]:
                continue
            if got is None:
                status[i], self.lens[c] = 1, 0
                continue
            full = self.lens[p] // PAGE
            for k in range(full):
                page = self.table[c][k] = self.table[p][k]
                if 0 <= page < len(self.refs):
                    self.refs[page] += 1
            if got:
                self.table[c][full] = got[0]
                self.refs[got[0]] = 1
                if cache is not None:
                    for a in cache.arrays():
                        a[got[0]] = a[self.table[p][full]]
            self.lens[c] = self.lens[p]
        return status

    def free(self, slots):
        for s in slots:
            if 0 <= s < len(self.lens):
                for k in range(min(pages_of(max(self.lens[s], 0)), len(self.table[s]))):
                    page = self.table[s][k]
                    if 0 <= page < len(self.refs):
                        self.refs[page] -= 1
                self.lens[s] = 0

    def compact(self, cache=None):
        live = sum(r > 0 for r in self.refs)
        src = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] <= 0]
        to = dict(zip(src, dst))
        for s, row in enumerate(self.table):
            for k in range(min(pages_of(max(self.lens[s], 0)), len(row))):
                row[k] = to.get(row[k], row[k])
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            if cache is not None:
                for x in cache.arrays():
                    x[b] = x[a]
        self.refs = [r if p < live else 0 for p, r in enumerate(self.refs)]
        return live


# ------------------------------------------------------------------ mixture of experts


def mx_weights(codes, scales, rows, K, fmt):
    """float64 [rows, K] of MX codes and MFMA-layout scale records."""
    if fmt == "mxfp4":
        w = np.empty((rows, K))
        lo, hi = codes & 15, codes >> 4
        w[:, 0::2] = E2M1[lo & 7] * np.where(lo & 8, -1, 1)
        w[:, 1::2] = E2M1[hi & 7] * np.where(hi & 8, -1, 1)
    else:
        w = E4M3[codes]
    r, kb = np.arange(rows)[:, None], np.arange(K)[None] // 32
    b = scales[r // 16, kb // 16 * 256 + 4 * (r % 16 + 16 * (kb % 4)) + kb % 16 // 4].astype(int)
    return np.where(b == 255, np.nan, w * 2.0 ** (b - 127.0))


def route(logits, topk, renormalize):
    """ids, weights of float64 logits [T, E] as moe_few_tokens states them."""
    T, E = logits.shape
    x = np.where(np.isnan(logits), -np.inf, logits)
    ids = np.array([sorted(range(E), key=lambda e, t=t: (-x[t, e], e))[:topk] for t in range(T)])
    w = np.zeros((T, topk))
    for t in range(T):
        top = x[t].max()
        if top == -np.inf:
            continue

        def share(v):
            return np.where(v == top, 1.0, np.where(v == -np.inf, 0.0, np.exp(
                np.where(np.isfinite(v), v, 0.0) - (top if np.isfinite(top) else 1e9))))
        own = share(x[t, ids[t]])
        w[t] = own / (own.sum() if renormalize else share(x[t]).sum())
    return ids.astype(np.int32), w


def moe(x, ids, weights, w1, w3, w2):
    """(y, bound): w1(e), w3(e), w2(e) give an expert's matrices.

    Bound: fp32 sums of H (and I) exact products, 2^-24 of their magnitudes a term; the gate
    within 2^-20 of itself; h kept to 16 bits (2^-16); weights 2^-22; y rounded to BF16."""
    T, H = x.shape
    y, b = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(ids.shape[1]):
            e, w = int(ids[t, j]), float(weights[t, j])
            if w == 0.0 or w1(e) is None:
                continue
            A, B, C = w1(e), w3(e), w2(e)
            I = A.shape[0]
            g, u = A @ x[t], B @ x[t]
            eg = (H + 8) * 2.0 ** -24 * (np.abs(A) @ np.abs(x[t]))
            eu = (H + 8) * 2.0 ** -24 * (np.abs(B) @ np.abs(x[t]))
            sg = g / (1 + np.exp(-g))
            h = sg * u
            eh = 1.1 * np.abs(u) * eg + np.abs(sg) * eu + 1.1 * eg * eu + np.abs(h) * (2.0 ** -20 + 2.0 ** -16)
            y[t] += w * (C @ h)
            b[t] += abs(w) * (np.abs(C) @ (eh + (2 * I + 32) * 2.0 ** -24 * (np.abs(h) + eh)))
            b[t] += abs(w) * 2.0 ** -20 * np.abs(C) @ np.abs(h)
    return y, (b + np.abs(y) * 2.0 ** -8) * (1 + 2.0 ** -7) + 2.0 ** -133


def bf16(x):
    """float64 array of the BF16 values nearest to x."""
    return torch.as_tensor(np.asarray(x, np.float64)).to(torch.bfloat16).double().numpy()
