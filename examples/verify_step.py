"""Steps of a decoder layer that verify trees of drafted tokens.

The layer of decode_step.py with queries and keys normalised and rotated, a sigmoid router with a
bias and groups, and a window with first tokens that stay visible.  A prompt's experts go through
the grouped quantizer and GEMM, their rows grouped on the device; a step's through the few-token
layer.  Each step drafts a tree for every sequence, whose first level are the likeliest tokens of
the step before, verifies it in one pass, keeps the path that the layer itself would have taken,
and writes that path's tokens over the tree's.  Weights are random; what the run shows is that the
operators fit together, eagerly and as a captured graph.

    python examples/verify_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import decode_step  # noqa: E402
from decode_step import MFMA, bsq, ints  # noqa: E402

# a tree of 7 drafted tokens: each node's parent, -1 for the sequence's last token
PARENTS = [-1, -1, 0, 0, 1, 2, 2]


def tree_masks(parents):
    """The words of a tree's masks (bit j: the node sees node j), and its nodes' depths."""
    masks, depth = [], []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return masks, depth


class Layer(decode_step.Layer):
    """`window` tokens and `sinks` first ones are seen."""

    def __init__(self, window=96, sinks=4, seed=0, **kw):
        super().__init__(seed=seed, **kw)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.window, self.sinks, d = window, sinks, self.dim
        self.q_weight, self.k_weight = 1 + 0.1 * torch.randn((2, d), generator=g, device="cuda")
        self.inv_freq = 10000.0 ** (-2 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d)
        self.bias = 0.05 * torch.randn(self.experts, generator=g, device="cuda")
        self.numbers = ints(range(self.experts))

    def route(self, x):
        return bsq.moe_route(x.float() @ self.router, self.topk, score="sigmoid", bias=self.bias, num_groups=4,
                             topk_groups=2, group_top=2, factor=2.0)

    def many_experts(self, x, ids, weights):
        """The layer that moe_few_tokens computes, for any number of tokens."""
        T, E, H = x.shape[0], self.experts, x.shape[1]
        w13, s13, w2, s2 = self.moe
        inter, n, most = w13.shape[0] // (2 * E), T * self.topk, T * self.topk // 16 * 16 + E * 16
        rows, scales, index, entry = bsq.moe_group_rows(ids, E, pad=16)

        def product(a, codes, b_scales, gather, fmt="mxfp4"):
            q, s = bsq.grouped_quantize_block_scaled(a, fmt, rows, scales, self.numbers, None, n, most,
                                                     row_indices=gather, scale_layout=MFMA)
            return bsq.grouped_block_scaled_matmul_mfma(q, s, rows, scales, self.numbers, n, most, codes,
                                                        b_scales, E, fmt, a.shape[1])
        a = product(x, w13, s13, index)
        h = torch.nn.functional.silu(a[:, :inter]) * a[:, inter:]
        y = product(h.to(torch.bfloat16), w2, s2, None)
        return (y[entry.long()] * weights[..., None]).sum(1).view(T, H).to(torch.bfloat16)

    def forward(self, tokens, offsets, max_rows, positions, masks=None):
        """Logits of the rows, and their keys and values."""
        x = self.embed[tokens]
        y = self.qkv(x).view(-1, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q, k, v = bsq.qk_norm_rope(q, k, positions, self.inv_freq, v=v, q_weight=self.q_weight,
                                   k_weight=self.k_weight)
        bsq.kv_cache_append(self.cache, k, v, offsets, self.lens, self.table, max_rows)
        a = bsq.kv_cache_attention_masked(q, self.cache, offsets, self.lens, self.table, max_rows,
                                          self.width * bsq.KV_PAGE, masks=masks, window=self.window,
                                          sinks=self.sinks)
        x = x + self.o(a.view(a.shape[0], -1)).to(torch.bfloat16)
        ids, weights = self.route(x)
        if x.shape[0] <= 64:
            m, _, _ = bsq.moe_few_tokens(x, "mxfp4", *self.moe, self.experts, self.topk, topk_ids=ids,
                                         topk_weights=weights)
        else:
            m = self.many_experts(x, ids, weights)
        return (x + m).float() @ self.embed.t().float(), k, v

    def take_back(self, slot, tokens):
        """The last tokens of a sequence: gone, with the pages that held nothing else."""
        length = int(self.lens[slot])
        for p in range(-(-(length - tokens) // bsq.KV_PAGE), -(-length // bsq.KV_PAGE)):
            self.refs[int(self.table[slot, p])] -= 1
        self.lens[slot] = length - tokens


class Verify:
    """A tree for every slot, as a graph over fixed buffers."""

    def __init__(self, layer, parents):
        masks, depth = tree_masks(parents)
        S, n = layer.slots, len(parents)
        self.layer, self.n = layer, n
        self.tokens = torch.zeros(S * n, dtype=torch.int32, device="cuda")
        self.add, self.all = ints([0] * S), ints(range(S))
        self.offsets, self.depth = ints(range(0, S * n + 1, n)), ints(depth)
        self.masks = torch.tensor(masks * S, dtype=torch.int64, device="cuda")[:, None]
        self.graph = None

    def eager(self):
        layer = self.layer
        layer.reserve(self.all, self.add)
        places = (layer.lens[:, None] - self.n + self.depth[None]).view(-1).to(torch.int32)
        logits, k, v = layer.forward(self.tokens, self.offsets, self.n, places, self.masks)
        return logits, k, v, bsq.token_logprobs(logits, top=2)

    def capture(self):
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = self.eager()

    def __call__(self, tokens):
        self.tokens.copy_(ints(tokens))
        self.add.fill_(self.n)
        if self.graph is None:
            return self.eager()
        self.graph.replay()
        logits, k, v, top = self.out
        return logits.clone(), k.clone(), v.clone(), type(top)(None, *(t.clone() for t in top[1:]))


def run(steps=4, seed=0, captured=True, slots=3):
    """Returns for each step its logits, and for each slot the tokens taken."""
    layer = Layer(seed=seed, slots=slots)
    g = torch.Generator().manual_seed(seed)
    lengths = [70, 5, 64][:slots]
    assert not layer.reserve(ints(range(slots)), ints(lengths)).any()
    offsets = ints([sum(lengths[:s]) for s in range(slots + 1)])
    places = torch.cat([ints(range(n)) for n in lengths])
    prompt = torch.randint(0, 512, (sum(lengths),), generator=g).to(torch.int32).cuda()
    logits, _, _ = layer.forward(prompt, offsets, max(lengths), places)
    last = bsq.token_logprobs(logits[offsets[1:].long() - 1], top=2)
    best, verify = last.top_ids.tolist(), Verify(layer, PARENTS)
    n, seen, taken = len(PARENTS), [], [[] for _ in range(slots)]
    for i in range(steps):
        if captured and i == 1:      # nothing drafted: the warm-up lengthens no sequence
            verify.add.zero_()
            verify.capture()
        drafts = torch.randint(0, 512, (slots, n), generator=g).tolist()
        for s in range(slots):
            drafts[s][0], drafts[s][1] = best[s]
        logits, k, v, top = verify(sum(drafts, []))
        seen.append(logits)
        wanted = top.top_ids.view(slots, n, 2).tolist()
        for s in range(slots):
            # the path of nodes whose tokens are those that the layer gives after their parents
            path, want = [], best[s]
            while True:
                node = [j for j in range(n) if PARENTS[j] == (path[-1] if path else -1) and drafts[s][j] == want[0]]
                if not node:
                    break
                path.append(node[0])
                want = wanted[s][node[0]]
            best[s] = want
            taken[s] += [drafts[s][j] for j in path]
            layer.take_back(s, n)
            rows = ints([s * n + j for j in path]).long()
            assert not layer.reserve(ints([s]), ints([len(path)])).any()
            owned = ints([0] * (s + 1) + [len(path)] * (slots - s))
            bsq.kv_cache_append(layer.cache, k[rows], v[rows], owned, layer.lens, layer.table, len(path))
    return layer, seen, taken


def main():
    layer, seen, taken = run()
    _, eager, same = run(captured=False)
    for i, (a, b) in enumerate(zip(seen, eager)):
        print(f"step {i}: trees of {len(PARENTS)} verified, captured equals eager: {torch.equal(a, b)}")
        assert torch.equal(a, b)
    print("tokens taken:", taken, "lengths:", layer.lens.tolist())
    assert taken == same


if __name__ == "__main__":
    main()
