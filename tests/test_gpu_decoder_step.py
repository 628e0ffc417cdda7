"""The operators of bsq_decoder.h together: the example's verified trees, captured calls whose
replays equal the eager results, calls on other streams, from several threads and of other
devices, and calls that find no memory."""
import os
import sys
import threading

import numpy as np
import pytest
import torch

import decoder_ref as R
from conftest import ROOT
from test_gpu_serving_kv import bsq, dev_cache, dev_rows, i32, make  # noqa: F401

pytestmark = pytest.mark.gpu


def test_example_verify_step(bsq):  # noqa: F811
    """Steps as a graph equal those without one; the likeliest drafted token is always taken."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import verify_step as ex

    layer, seen, taken = ex.run(steps=5, seed=2)
    _, eager, same = ex.run(steps=5, seed=2, captured=False)
    assert len(seen) == 5 and all(torch.isfinite(x).all() for x in seen)
    assert taken == same and all(torch.equal(a, b) for a, b in zip(seen, eager))
    assert all(len(t) >= 5 for t in taken)
    assert layer.lens.tolist() == [n + len(t) for n, t in zip((70, 5, 64), taken)]
    used = sum(-(-n // 64) for n in layer.lens.tolist())
    assert int(layer.refs.sum()) == used and int((layer.refs == 1).sum()) == used


def test_tree_step_is_the_chains_of_its_paths(bsq):  # noqa: F811
    """Norm, rotation, append and attention of a tree: a node's row is what its path gives when its
    tokens are appended one behind the other (values of one size: no page's scale changes)."""
    import serving_ref as S

    rng = np.random.default_rng(5)
    n, before, heads, hq, D = 9, 100, 2, 4, 64
    parents = [-1, 0, 0, 1, 1, 2, -1, 6, 3]
    masks = [set() for _ in range(n)]
    for i, p in enumerate(parents):
        masks[i] = (masks[p] if p >= 0 else set()) | {i}
    depth = [len(m) - 1 for m in masks]
    x = torch.tensor(np.sign(rng.standard_normal((before + n, hq + 2 * heads, D))) *
                     rng.uniform(0.5, 1, (before + n, hq + 2 * heads, D)), device="cuda").float()
    f = torch.tensor(100.0 ** (-np.arange(16) / 16), device="cuda")

    def run(rows, places, tree=None):
        c = bsq.kv_cache(3, heads, D)
        q, k, v = x[rows].split([hq, heads, heads], 1)
        q, k, v = bsq.qk_norm_rope(q, k, i32(places), f, v=v)
        L, t = len(rows), i32([[2, 0, 1]])
        bsq.kv_cache_append(c, k, v, i32([0, L]), i32([L]), t, L)
        last = L - before
        w = None if tree is None else torch.tensor(R.words(tree, 1), device="cuda")
        return bsq.kv_cache_attention_masked(q[before:], c, i32([0, last]), i32([L]), t, last, L, masks=w)

    first = list(range(before))
    tree = run(first + [before + i for i in range(n)], first + [before + d for d in depth], masks)
    for i in range(n):
        path = sorted(masks[i])
        chain = run(first + [before + j for j in path], first + [before + d for d in range(len(path))])
        torch.cuda.synchronize()
        # both are off by what the reference's bounds allow: half a step of BF16 and 2^-10 of the values
        assert torch.allclose(tree[i].float(), chain[-1].float(), rtol=2 ** -7, atol=2 ** -9), i
    assert S.PAGE == 64


# ------------------------------------------------------------------ graphs, streams, threads


NAMES = ["rope", "tree", "tree split", "sinks", "route", "rows", "many rows", "logprobs", "logprobs join"]


class Call:
    """One operator: call(stream) gives new outputs from inputs that stay as they are."""

    def __init__(self, bsq, name, seed=0):  # noqa: F811
        rng = np.random.default_rng(len(name) + seed)

        def rand(*shape):
            return torch.tensor(rng.standard_normal(shape), device="cuda").float()
        if name == "rope":
            q, k, v = rand(33, 8, 64).split([4, 2, 2], 1)
            p, f, w = i32(rng.integers(0, 9999, 33)), torch.tensor(0.9 ** np.arange(32), device="cuda"), rand(64)
            self.call = lambda s: bsq.qk_norm_rope(q, k, p, f, v=v, q_weight=w, k_weight=w, stream=s)
        elif name in ("tree", "tree split", "sinks"):
            lens, rows = ([9000, 70] if "split" in name else [200, 70]), [9, 5]
            c, q, off, table = make(3, lens, rows, 2, 8, 64)
            masks = None
            kw = dict(sinks=5, window=60)
            if name != "sinks":
                masks, kw = torch.tensor(R.words(R.random_tree(rng, 9) + R.random_tree(rng, 5), 1), device="cuda"), {}
            d, a = dev_cache(bsq, c), (i32(off), i32(lens), i32(table), 9, max(lens))
            q = dev_rows(q)
            self.call = lambda s: bsq.kv_cache_attention_masked(q, d, *a, masks=masks, return_lse=True, stream=s, **kw)
        elif name == "route":
            z, b = rand(50, 64), 0.1 * rand(64)
            self.call = lambda s: bsq.moe_route(z, 6, score="sigmoid", bias=b, num_groups=8, topk_groups=3,
                                                group_top=2, stream=s)
        elif name.endswith("rows"):
            ids = i32(rng.integers(0, 70, (2000 if "many" in name else 60, 5)))
            self.call = lambda s: bsq.moe_group_rows(ids, 70, stream=s)
        else:
            z = rand(7, 40000 if "join" in name else 900)
            t = i32(rng.integers(0, 900, (7, 2)))
            self.call = lambda s: bsq.token_logprobs(z, t, top=9, stream=s)
        torch.cuda.synchronize()
        self.want = [t.clone() for t in self.call(None)]
        torch.cuda.synchronize()

    def right(self, got):
        return all(torch.equal(a, b) for a, b in zip(got, self.want))


def sleep():
    torch.cuda._sleep(20_000_000)


@pytest.mark.parametrize("name", NAMES)
def test_captured_calls_replay(bsq, name):  # noqa: F811
    """Two graphs of a call that are replayed in turn, with eager calls between."""
    c, other = Call(bsq, name), Call(bsq, name, seed=1)
    graphs = []
    for x in (c, other):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = x.call(None)
        graphs.append((x, graph, got))
    for _ in range(4):
        for x, graph, got in graphs:
            for t in got:
                t.fill_(9)
            graph.replay()
        torch.cuda.synchronize()
        assert all(x.right(got) for x, _, got in graphs)
        assert c.right(c.call(None)) and other.right(other.call(None))
        torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["tree split", "many rows", "logprobs join"])
def test_graphs_that_share_a_workspace(bsq, name):  # noqa: F811
    """A caller's workspace, which two captured calls use one after the other."""
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    calls = [Call(bsq, name, seed) for seed in (0, 1)]
    fn = {"tree split": "kv_cache_attention_masked", "many rows": "moe_group_rows", "logprobs join": "token_logprobs"}[name]
    real, graphs = getattr(bsq, fn), []
    setattr(bsq, fn, lambda *a, **kw: real(*a, workspace=ws, **kw))
    try:
        for c in calls:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                got = c.call(None)
            graphs.append((graph, got))
    finally:
        setattr(bsq, fn, real)
    for _ in range(3):
        ws.fill_(255)
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(c.right(got) for c, (_, got) in zip(calls, graphs))


@pytest.mark.parametrize("name", NAMES)
def test_other_streams(bsq, name):  # noqa: F811
    """Calls on the current stream and two others in turn, each stream's outputs and workspaces its
    own; dropped outputs of a call that has not run are not given to the current stream."""
    c, streams = Call(bsq, name), [None, torch.cuda.Stream(), torch.cuda.Stream()]
    got = [c.call(s) for _ in range(6) for s in streams]
    torch.cuda.synchronize()
    assert all(c.right(g) for g in got)
    with torch.cuda.stream(streams[1]):
        sleep()
    got = c.call(streams[1])
    asleep = torch.cuda.Event()
    asleep.record(streams[1])
    kept, places = got[0], {t.data_ptr(): t.nbytes for t in got[1:]}
    shapes = [(t.shape, t.dtype) for t in got[1:]]
    del got
    mine = [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes for _ in range(3)]
    assert not asleep.query()
    for t in mine:
        for p, n in places.items():
            assert t.data_ptr() + t.nbytes <= p or p + n <= t.data_ptr()
    torch.cuda.synchronize()
    assert torch.equal(kept, c.want[0])


def test_threads_on_their_own_streams(bsq):  # noqa: F811
    """All operators at once from a thread each; one thread's refused calls leave the others alone."""
    calls, errors = [Call(bsq, n) for n in NAMES], []

    def work(c):
        try:
            stream = torch.cuda.Stream()
            got = []
            for _ in range(10):
                with pytest.raises(bsq.BsqError, match="top="):
                    bsq.token_logprobs(torch.zeros((1, 3), device="cuda"), top=9, stream=stream)
                got.append(c.call(stream))
            stream.synchronize()
            if not all(c.right(g) for g in got):
                errors.append("wrong")
        except BaseException as e:                           # reported on the main thread
            errors.append(repr(e))
    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=100)
    assert not errors and not any(t.is_alive() for t in threads)


def test_outputs_that_c_callers_leave_out(bsq):  # noqa: F811
    """NULL for v, entry_rows, entropy and the tokens, with the raw library: the other outputs stay."""
    raw, g = bsq.serving_lib(), torch.Generator(device="cuda").manual_seed(1)
    torch.cuda.synchronize()
    for T in (30, 3000):
        ids = torch.randint(0, 50, (T, 4), generator=g, device="cuda", dtype=torch.int32)
        want = bsq.moe_group_rows(ids, 50, pad=16)
        got = [torch.full_like(t, -9) for t in want[:3]]
        ws = torch.empty(max(raw.moe_group_rows_workspace(T, 4, 50), 16), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert raw.moe_group_rows(ids.data_ptr(), T, 4, 50, 16, *(t.data_ptr() for t in got), None, ws.data_ptr(),
                                  ws.numel(), None) == 0
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for V in (700, 30000):
        z = torch.randn((3, V), generator=g, device="cuda")
        want = bsq.token_logprobs(z, top=4)
        ids, best = torch.full_like(want.top_ids, -9), torch.full_like(want.top_logprobs, -9)
        ws = torch.empty(max(raw.token_logprobs_workspace(3, V, 4), 16), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert raw.token_logprobs(1, z.data_ptr(), V, 3, V, None, 0, 4, None, None, ids.data_ptr(), best.data_ptr(),
                                  ws.data_ptr(), ws.numel(), None) == 0
        torch.cuda.synchronize()
        assert torch.equal(ids, want.top_ids) and torch.equal(best, want.top_logprobs)
    x = torch.randn((5, 3, 64), generator=g, device="cuda")
    q, k = torch.empty((2, 5, 64), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    assert raw.qk_norm_rope(1, x.data_ptr(), 192, 1, x.data_ptr() + 256, 192, 1, None, 0, 64, 5, None, None, 0.0, None,
                            None, 0, 0, q.data_ptr(), 64, k.data_ptr(), 64, None, 0, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(q, x[:, 0].to(q.dtype)) and torch.equal(k, x[:, 1].to(k.dtype))


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_another_device(bsq, name):  # noqa: F811
    with torch.cuda.device(1):
        c = Call(bsq, name)
    got = c.call(None)
    torch.cuda.synchronize(1)
    assert torch.cuda.current_device() == 0 and got[0].device.index == 1 and c.right(got)


def test_out_of_memory_is_torchs_error(bsq):  # noqa: F811
    z = torch.zeros((1 << 20, 16), device="cuda")
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total, held = torch.cuda.get_device_properties(0).total_memory, []
    try:
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (32 << 20)) / total)
        with pytest.raises(torch.OutOfMemoryError):
            for _ in range(10000):
                held.append(torch.empty_like(z))
        with pytest.raises(torch.OutOfMemoryError):
            bsq.moe_route(z, 16)
    finally:
        del held
        torch.cuda.set_per_process_memory_fraction(1.0)
    ids, w = bsq.moe_route(z, 16)
    torch.cuda.synchronize()
    assert bool((ids == torch.arange(16, device="cuda")).all()) and bool((w == 1 / 16).all())
