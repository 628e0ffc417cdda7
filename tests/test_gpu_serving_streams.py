"""Calls on another stream than the current one: their outputs and workspaces are that stream's
memory, so neither stream's work overwrites the other's, however the calls interleave and
whatever of their results is dropped."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_serving_kv import bsq, dev_cache, dev_rows, i32, make  # noqa: F401
from test_gpu_serving_moe import Layer

pytestmark = pytest.mark.gpu

NAMES = ["attention", "attention split", "experts", "few experts", "compact", "reserve", "fork"]


class Call:
    """One operator: call(stream) gives new outputs from inputs that stay as they are."""

    def __init__(self, bsq, name):
        rng = np.random.default_rng(len(name))
        if name.startswith("attention"):
            lens = [9000, 70] if name.endswith("split") else [130, 70]
            c, q, off, table = make(3, lens, [2, 1], 2, 8, 64)
            d, a = dev_cache(bsq, c), (i32(off), i32(lens), i32(table), 2, max(lens))
            q = dev_rows(q)
            self.call = lambda s: bsq.kv_cache_attention(q, d, *a, return_lse=True, stream=s)
        elif name.endswith("experts"):
            T = 2 if name.startswith("few") else 20
            L = Layer(T, 9, 256, 128, "mxfp4")
            w, x = L.dev(), dev_rows(R.bf16(rng.standard_normal((T, 256))))
            lg = torch.from_numpy(rng.standard_normal((T, 9)).astype(np.float32)).cuda()
            self.call = lambda s: bsq.moe_few_tokens(x, "mxfp4", *w, 9, 2, router_logits=lg, stream=s)
        else:
            P, S, M = 900, 4, 60
            d = bsq.kv_cache(P, 1, 64)
            refs = i32([1] * 30 + [0] * 100 + [1] * 20 + [0] * (P - 150))
            table, lens = i32(np.arange(S * M).reshape(S, M)), i32([64, 70, 0, 0])
            one, two, add = i32([0, 1]), i32([2, 3]), i32([64, 640])
            # inputs that a call changes are copied on the call's stream
            if name == "compact":
                def call(s):
                    return bsq.kv_pages_compact(d, table, lens, refs, stream=s)
            else:
                def call(s):
                    with torch.cuda.stream(s):
                        t, n, r = table.clone(), lens.clone(), refs.clone()
                    if name == "fork":
                        return (bsq.kv_pages_fork(d, t, n, r, one, two, stream=s), t, n, r)
                    return (bsq.kv_pages_reserve(t, n, r, one, add, stream=s), t, n, r)
            self.call = call
        torch.cuda.synchronize()
        self.want = [t.clone() for t in self.call(torch.cuda.current_stream())]
        torch.cuda.synchronize()

    def right(self, got):
        return all(torch.equal(a, b) for a, b in zip(got, self.want))


def sleep():
    """Some milliseconds of the current stream."""
    torch.cuda._sleep(20_000_000)


def sizes_of(call):
    """Bytes of every block that the call allocates, its workspace among them."""
    torch.cuda.synchronize()
    torch.cuda.memory._record_memory_history(max_entries=10000)
    try:
        out = call(torch.cuda.current_stream())
        torch.cuda.synchronize()
        trace = torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    del out
    return [e["size"] for e in trace if e["action"] == "alloc"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_reads(bsq, name):  # noqa: F811
    """Blocks of the call's own sizes, freed behind queued work of the current stream, are not
    what a call on another stream writes to."""
    c, side = Call(bsq, name), torch.cuda.Stream()
    sizes = sizes_of(c.call)
    assert sizes
    xs = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    ys = [torch.empty_like(x) for x in xs]
    torch.cuda.synchronize()
    sleep()
    for x, y in zip(xs, ys):
        y.copy_(x)
    del xs, x
    got = c.call(side)
    torch.cuda.synchronize()
    assert all(bool((y == 3).all()) for y in ys)
    assert c.right(got)


@pytest.mark.parametrize("name", NAMES)
def test_dropped_outputs_stay_with_their_stream(bsq, name):  # noqa: F811
    """What a call on another stream returned and nobody kept is not given to the current stream
    while the call has not run yet."""
    c, side = Call(bsq, name), torch.cuda.Stream()
    with torch.cuda.stream(side):
        sleep()
    got = c.call(side)
    asleep = torch.cuda.Event()
    asleep.record(side)
    kept, dropped = got[0], got[1:]
    places = {t.data_ptr(): t.nbytes for t in dropped}
    shapes = [t.shape for t in dropped]
    del got, dropped
    mine = [torch.full(s, -1, dtype=d, device="cuda") for s in shapes for d in (torch.int32, torch.float32)
            for _ in range(3)]
    assert not asleep.query()
    for t in mine:
        for p, n in places.items():
            assert t.data_ptr() + t.nbytes <= p or p + n <= t.data_ptr()
    torch.cuda.synchronize()
    assert torch.equal(kept, c.want[0])


@pytest.mark.parametrize("name", NAMES)
def test_outputs_that_the_callers_stream_still_reads(bsq, name):  # noqa: F811
    """Outputs of a call on another stream, read by the current one behind other work and dropped:
    the next call on that stream gets other memory."""
    c, side = Call(bsq, name), torch.cuda.Stream()
    first = c.call(side)[0]
    torch.cuda.current_stream().wait_stream(side)
    sleep()
    copy = torch.empty_like(first)
    copy.copy_(first)
    asleep = torch.cuda.Event()
    asleep.record()
    place = first.data_ptr()
    del first
    again = [c.call(side) for _ in range(3)]
    assert not asleep.query()
    assert all(a[0].data_ptr() != place for a in again)
    torch.cuda.synchronize()
    assert torch.equal(copy, c.want[0]) and all(c.right(a) for a in again)


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_without_waiting(bsq, name):  # noqa: F811
    """Independent calls, on the current stream and two others in turn, whose workspaces go back at
    each return."""
    c, streams = Call(bsq, name), [None, torch.cuda.Stream(), torch.cuda.Stream()]
    now = torch.cuda.current_stream()
    got = [c.call(s or now) for _ in range(8) for s in streams]
    torch.cuda.synchronize()
    assert all(c.right(g) for g in got)


def test_another_stream_in_a_captured_graph(bsq):  # noqa: F811
    """A call forked to another stream inside a capture: every replay gives the eager result."""
    c, side = Call(bsq, "attention split"), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        now = torch.cuda.current_stream()
        side.wait_stream(now)
        got = c.call(side)
        now.wait_stream(side)
    for _ in range(4):
        for t in got:
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert c.right(got)
        assert c.right(c.call(torch.cuda.current_stream()))
        torch.cuda.synchronize()


def test_current_stream_and_device_after_a_call(bsq):  # noqa: F811
    """A call on another stream, and one that is refused there, leave the current one current."""
    c, side, now = Call(bsq, "attention"), torch.cuda.Stream(), torch.cuda.current_stream()
    c.call(side)
    assert torch.cuda.current_stream() == now
    d, q = bsq.kv_cache(3, 1, 64), torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bsq.BsqError):
        bsq.kv_cache_attention(q, d, i32([0, 1]), i32([0]), i32([[0]]), 1, 1, window=-1, stream=side)
    assert torch.cuda.current_stream() == now and torch.cuda.current_device() == 0
    torch.cuda.synchronize()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_of_another_device(bsq):  # noqa: F811
    """Tensors of a device that is not the current one: the call runs there."""
    with torch.cuda.device(1):
        c = Call(bsq, "attention")
    now = torch.cuda.current_device()
    got = c.call(None)
    torch.cuda.synchronize(1)
    assert now == torch.cuda.current_device() and got[0].device.index == 1 and c.right(got)
