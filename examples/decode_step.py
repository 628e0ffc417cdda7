"""A decoder layer served from block-scaled state and weights.

Projections are MXFP8 matrix products, the key/value cache is paged E4M3, the experts are
MXFP4: prompts go through in chunks, each sequence is forked into two samples, a captured graph
replays the decode step, finished samples give their pages back and the pool is compacted while
the others go on.  Weights are random; what the run shows is that the operators fit together:
a sample that is fed the same tokens as its sibling gives the same bits, before and after its
pages move, eagerly and from the graph.

    python examples/decode_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fp8_quantization_amd as bsq  # noqa: E402

MFMA = bsq.SCALES_MFMA16


class Linear:
    """y = x W^T in MXFP8: weights quantized once, activations on the way."""

    def __init__(self, rows, width, generator):
        w = torch.randn((rows, width), generator=generator, device="cuda") * width ** -0.5
        self.codes, self.scales = bsq.quantize_block_scaled(w.to(torch.bfloat16), "mxfp8",
                                                            scale_layout=MFMA)
        self.width = width

    def __call__(self, x):
        q, s = bsq.quantize_block_scaled(x, "mxfp8", scale_layout=MFMA)
        return bsq.block_scaled_matmul_mfma(q, s, self.codes, self.scales, "mxfp8", self.width)


class Layer:
    """Attention over the paged cache and a mixture of experts, for `slots` sequences."""

    def __init__(self, slots=8, pages=64, hidden=256, heads=4, kv_heads=2, dim=64, experts=8, topk=2,
                 inter=128, vocab=512, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.experts, self.topk, self.slots = experts, topk, slots
        self.embed = torch.randn((vocab, hidden), generator=g, device="cuda").to(torch.bfloat16)
        self.qkv = Linear((heads + 2 * kv_heads) * dim, hidden, g)
        self.o = Linear(hidden, heads * dim, g)
        self.router = torch.randn((hidden, experts), generator=g, device="cuda") * hidden ** -0.5
        self.moe = []
        for rows, width in ((experts * 2 * inter, hidden), (experts * hidden, inter)):
            w = torch.randn((rows, width), generator=g, device="cuda") * width ** -0.5
            self.moe += bsq.quantize_block_scaled(w.to(torch.bfloat16), "mxfp4", scale_layout=MFMA)
        self.cache = bsq.kv_cache(pages, kv_heads, dim)
        self.width = 8                                       # pages a sequence may have
        self.table = torch.zeros((slots, self.width), dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(slots, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")

    def forward(self, tokens, offsets, max_rows):
        """Logits of the rows; `offsets` deals them to the slots, whose lengths count them."""
        x = self.embed[tokens]
        y = self.qkv(x).to(torch.bfloat16).view(-1, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], 1)
        bsq.kv_cache_append(self.cache, k, v, offsets, self.lens, self.table, max_rows)
        a = bsq.kv_cache_attention(q, self.cache, offsets, self.lens, self.table, max_rows,
                                   self.width * bsq.KV_PAGE)
        x = x + self.o(a.view(a.shape[0], -1)).to(torch.bfloat16)
        m, _, _ = bsq.moe_few_tokens(x, "mxfp4", *self.moe, self.experts, self.topk,
                                     router_logits=x.float() @ self.router)
        return (x + m).float() @ self.embed.t().float()

    def reserve(self, slots, tokens):
        return bsq.kv_pages_reserve(self.table, self.lens, self.refs, slots, tokens)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prompts(layer, texts, chunk=24):
    """Run the prompts (slot -> tokens) through the layer, `chunk` rows a sequence at a time."""
    logits = {}
    for at in range(0, max(map(len, texts.values())), chunk):
        part = {s: t[at:at + chunk] for s, t in texts.items() if t[at:at + chunk]}
        ok = layer.reserve(ints(list(part)), ints([len(t) for t in part.values()]))
        assert not ok.any(), "the pool is too small"
        rows = [len(part.get(s, [])) for s in range(layer.slots)]
        offsets = ints([sum(rows[:s]) for s in range(layer.slots + 1)])
        out = layer.forward(ints([t for s in sorted(part) for t in part[s]]), offsets, chunk)
        for s in part:
            logits[s] = out[offsets[s + 1] - 1]
    return logits


class Step:
    """One token for every slot in use: the whole step as a graph over fixed buffers.
    Slots out of use own a row too; with length 0 they see nothing, and reserve adds nothing."""

    def __init__(self, layer):
        self.layer = layer
        self.tokens = torch.zeros(layer.slots, dtype=torch.int32, device="cuda")
        self.add = torch.zeros(layer.slots, dtype=torch.int32, device="cuda")
        self.all = ints(list(range(layer.slots)))
        self.offsets = ints(list(range(layer.slots + 1)))
        self.graph = None

    def eager(self):
        self.layer.reserve(self.all, self.add)
        return self.layer.forward(self.tokens, self.offsets, 1)

    def capture(self):
        """With `add` 0 the warm-up neither lengthens a sequence nor writes a new token."""
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.logits = self.eager()

    def __call__(self, tokens, add):
        self.tokens.copy_(ints(tokens))
        self.add.copy_(ints(add))
        if self.graph is None:
            return self.eager()
        self.graph.replay()
        return self.logits.clone()


def run(steps=6, seed=0):
    """Returns the logits of every decode step, by slot."""
    layer = Layer(seed=seed)
    g = torch.Generator().manual_seed(seed)
    texts = {s: torch.randint(0, 512, (n,), generator=g).tolist() for s, n in ((0, 70), (1, 64), (2, 5))}
    first = prompts(layer, texts)
    # two samples of each: slots 4, 5, 6
    ok = bsq.kv_pages_fork(layer.cache, layer.table, layer.lens, layer.refs, ints([0, 1, 2]), ints([4, 5, 6]))
    assert not ok.any()
    live = [0, 1, 2, 4, 5, 6]
    token = [0] * layer.slots
    for s in (0, 1, 2):
        token[s] = token[s + 4] = int(first[s].argmax())
    step, seen = Step(layer), []
    for i in range(steps):
        if i == 1:
            step.capture()
        if i == 3:
            # two samples end; the pages of the rest move to the front of the pool
            bsq.kv_pages_free(layer.table, layer.lens, layer.refs, ints([0, 5]))
            live = [s for s in live if s not in (0, 5)]
            bsq.kv_pages_compact(layer.cache, layer.table, layer.lens, layer.refs,
                                 table_out=layer.table, refcounts_out=layer.refs)
        out = step(token, [int(s in live) for s in range(layer.slots)])
        seen.append({s: out[s] for s in live})
        for s in live:
            token[s] = int(out[s].argmax())
    return layer, seen


def main():
    layer, seen = run()
    for i, out in enumerate(seen):
        pairs = [(s, s + 4) for s in (0, 1, 2) if s in out and s + 4 in out]
        same = all(torch.equal(out[a], out[b]) for a, b in pairs)
        print(f"step {i}: {len(out)} samples, siblings equal: {same}")
        assert same
    used = int((layer.refs > 0).sum())
    print(f"pages in use: {used}, the first {used} of the pool: {bool((layer.refs[:used] > 0).all())}")


if __name__ == "__main__":
    main()
