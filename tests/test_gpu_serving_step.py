"""The operators together: the example's decoder layer, and a captured sequence of calls whose
replays equal the eager results."""
import os
import sys

import numpy as np
import pytest
import torch

import serving_ref as R
from conftest import ROOT
from test_gpu_serving_kv import bsq, dev_cache, dev_rows, i32, make  # noqa: F401
from test_gpu_serving_moe import Layer

pytestmark = pytest.mark.gpu


def test_example_decode_step(bsq):  # noqa: F811
    """Siblings give equal bits, eagerly, from the graph and after their pages moved; the graph's
    steps equal those of a run without one."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_step as ex

    layer, seen = ex.run(steps=6, seed=1)
    for out in seen:
        for s in (0, 1, 2):
            if s in out and s + 4 in out:
                assert torch.equal(out[s], out[s + 4])
            for t in (s, s + 4):
                assert t not in out or torch.isfinite(out[t]).all()
    used = int((layer.refs > 0).sum())
    assert bool((layer.refs[:used] > 0).all()) and sorted(seen[-1]) == [1, 2, 4, 6]
    capture, ex.Step.capture = ex.Step.capture, lambda self: None
    try:
        _, eager = ex.run(steps=6, seed=1)
    finally:
        ex.Step.capture = capture
    for a, b in zip(seen, eager):
        assert sorted(a) == sorted(b) and all(torch.equal(a[s], b[s]) for s in a)


@pytest.mark.parametrize("T", [2, 30])
def test_captured_calls_replay(bsq, T):  # noqa: F811
    """Append, attention (split over the tokens), fork, free, compaction and the experts in one
    graph, replayed with other eager work between; every replay equals the eager calls."""
    lens, rows = [5000, 130, 64], [1, 1, 1]
    c, q, off, table = make(T, lens, rows, 1, 4, 64, extra_pages=40)
    P, M = c.ks.shape[0], len(table[0])
    rng = np.random.default_rng(T)
    L = Layer(T, 6, 128, 128, "mxfp4")
    w = L.dev()
    x = dev_rows(R.bf16(rng.standard_normal((T, 128))))
    logits = torch.from_numpy(rng.standard_normal((T, 6)).astype(np.float32)).cuda()
    kv = dev_rows(R.bf16(rng.standard_normal((3, 2, 1, 64))))
    refs0 = np.zeros(P, int)
    for s, n in enumerate(lens):
        refs0[table[s][:R.pages_of(n)]] = 1
    table0 = i32(table + [[0] * M] * 2)
    lens0, refs0, qd = i32(lens + [0, 0]), i32(refs0), dev_rows(q)
    o5, start = i32(list(off) + [3, 3]), dev_cache(bsq, c)

    def fresh():
        return [t.clone() for t in start] + [table0.clone(), lens0.clone(), refs0.clone()]

    def calls(st):
        d, tb, ln, rf = bsq.KvCache(*st[:4]), *st[4:]
        bsq.kv_cache_append(d, kv[:, 0], kv[:, 1], o5, ln, tb, 1)
        out, lse = bsq.kv_cache_attention(qd, d, o5, ln, tb, 1, 5000, return_lse=True)
        ok = bsq.kv_pages_fork(d, tb, ln, rf, i1, i2)
        res = bsq.kv_pages_reserve(tb, ln, rf, i2, add)
        bsq.kv_pages_free(tb, ln, rf, i1)
        t2, r2, n = bsq.kv_pages_compact(d, tb, ln, rf)
        y, ids, ws = bsq.moe_few_tokens(x, "mxfp4", *w, 6, 2, router_logits=logits)
        return [out, lse, ok, res, r2, n, y, ids, ws, ln, t2[4, :2]]

    i1, i2, add = i32([0, 1]), i32([3, 4]), i32([70, 0])
    st = fresh()
    want = [t.clone() for t in calls(st)] + [t.clone() for t in st]
    st = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(st)
    for i in range(4):
        for a, b in zip(st, fresh()):
            a.copy_(b)
        for t in got[:9]:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got + st, want)):
            assert torch.equal(a, b), (i, k)
        calls(fresh())                                       # other work between replays
        torch.cuda.synchronize()
