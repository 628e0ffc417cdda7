"""moe_few_tokens on the GPU against the 64-bit reference within its rounding bounds; the
routing exactly."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_serving_kv import bsq, dev_rows, i32  # noqa: F401

pytestmark = pytest.mark.gpu


class Layer:
    """Random MX weights: device tensors and each expert's matrices in 64 bits."""

    def __init__(self, seed, E, H, I, fmt):
        rng = np.random.default_rng(seed)
        self.E, self.H, self.I, self.fmt = E, H, I, fmt
        self.host = {}
        for name, n, k in (("w13", 2 * I, H), ("w2", H, I)):
            if fmt == "mxfp4":
                codes = rng.integers(0, 256, (E * n, k // 2), dtype=np.uint8)
            else:
                codes = R.to_e4m3(rng.standard_normal((E * n, k)) * 3)
            # every byte of a record set: those past K are never used
            scales = rng.integers(118, 123, (E * n // 16, (k + 511) // 512 * 256), dtype=np.uint8)
            used = np.zeros_like(scales, dtype=bool)
            r, kb = np.arange(16)[:, None], np.arange(k // 32)[None]
            used[:, (kb // 16 * 256 + 4 * (r + 16 * (kb % 4)) + kb % 16 // 4).reshape(-1)] = True
            scales[~used] = 255
            self.host[name] = (codes, scales, n, k)
        self.dense = {}

    def dev(self):
        return [torch.from_numpy(a).cuda() for n in ("w13", "w2") for a in self.host[n][:2]]

    def matrix(self, name, e):
        if not 0 <= e < self.E:
            return None
        if (name, e) not in self.dense:
            codes, scales, n, k = self.host[name]
            self.dense[name, e] = R.mx_weights(codes[e * n:(e + 1) * n],
                                               scales[e * n // 16:(e + 1) * n // 16], n, k, self.fmt)
        return self.dense[name, e]

    def reference(self, x, ids, weights):
        def w1(e):
            m = self.matrix("w13", e)
            return None if m is None else m[:self.I]
        return R.moe(x, ids, weights, w1, lambda e: self.matrix("w13", e)[self.I:],
                     lambda e: self.matrix("w2", e))


def check(y, want, bound):
    y = y.double().cpu().numpy()
    assert np.all(np.abs(y - want) <= bound), np.max(np.abs(y - want) / bound)


def given(seed, T, E, k):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32) + 0.1
    return ids, w


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 1, 1, 128, 128), (1, 9, 8, 384, 256), (3, 40, 4, 640, 128), (4, 300, 16, 256, 128),
    (5, 6, 3, 256, 640), (16, 4, 4, 512, 384), (16, 33, 8, 128, 512), (17, 3, 1, 384, 128),
    (33, 5, 2, 256, 1152), (64, 2, 2, 128, 128), (64, 70, 1, 256, 256), (64, 20, 6, 768, 128)])
def test_routed_by_the_caller(bsq, fmt, T, E, k, H, I):  # noqa: F811
    L = Layer(T + E, E, H, I, fmt)
    x = R.bf16(np.random.default_rng(T).standard_normal((T, H)))
    ids, w = given(T * E, T, E, k)
    y, i2, w2 = bsq.moe_few_tokens(dev_rows(x), fmt, *L.dev(), E, k, topk_ids=i32(ids),
                                   topk_weights=torch.from_numpy(w).cuda())
    torch.cuda.synchronize()
    check(y, *L.reference(x, ids, w))
    assert torch.equal(i2.cpu(), torch.from_numpy(ids)) and torch.equal(w2.cpu(), torch.from_numpy(w))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,E,k,H,I", [
    (2, 20, 8, 128, 1664), (8, 16, 2, 640, 1536), (16, 200, 8, 128, 256), (64, 100, 2, 384, 256),
    (64, 24, 12, 128, 1024)])
def test_wide_tiles(bsq, fmt, T, E, k, H, I):  # noqa: F811
    """Columns of h enough for 32 a workgroup: few entries, a workgroup an entry or an expert, one
    block of entries and two."""
    L = Layer(T + E, E, H, I, fmt)
    x = R.bf16(np.random.default_rng(T).standard_normal((T, H)))
    ids, w = given(T * E, T, E, k)
    y, _, _ = bsq.moe_few_tokens(dev_rows(x), fmt, *L.dev(), E, k, topk_ids=i32(ids),
                                 topk_weights=torch.from_numpy(w).cuda())
    torch.cuda.synchronize()
    check(y, *L.reference(x, ids, w))
    logits = np.random.default_rng(E).standard_normal((T, E)).astype(np.float32)
    y, i2, w2 = bsq.moe_few_tokens(dev_rows(x), fmt, *L.dev(), E, k,
                                   router_logits=torch.from_numpy(logits).cuda())
    torch.cuda.synchronize()
    check(y, *L.reference(x, i2.cpu().numpy(), w2.cpu().numpy()))


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (2, 128, 8), (4, 129, 16), (5, 256, 8), (3, 1024, 5),
                                   (20, 65, 1), (64, 16, 4)])
def test_routed_by_logits(bsq, T, E, k, renormalize):  # noqa: F811
    rng = np.random.default_rng(T + E)
    L = Layer(E, E, 128, 128, "mxfp4") if E <= 300 else Layer(E, E, 128, 128, "mxfp8")
    x = R.bf16(rng.standard_normal((T, 128)))
    logits = (rng.standard_normal((T, E)) * 3).astype(np.float32)
    logits[0] = np.round(logits[0])                          # ties go to the lower expert
    y, ids, w = bsq.moe_few_tokens(dev_rows(x), L.fmt, *L.dev(), E, k,
                                   router_logits=torch.from_numpy(logits).cuda(),
                                   renormalize=renormalize)
    torch.cuda.synchronize()
    wi, ww = R.route(logits.astype(np.float64), k, renormalize)
    assert np.array_equal(ids.cpu().numpy(), wi)
    # an exponent of up to |x| log2 e is rounded at 2^-24 of itself, twice
    spread = logits.max() - logits.min()
    assert np.all(np.abs(w.double().cpu().numpy() - ww) <= ww * (spread + 8 + E) * 2.0 ** -22)
    check(y, *L.reference(x, wi, w.double().cpu().numpy()))


def test_logits_that_rule_experts_out(bsq):  # noqa: F811
    """-inf, NaN, +inf and rows of nothing: weight 0 and no use of such an expert's weights."""
    E, k, H, I = 6, 3, 256, 128
    L = Layer(1, E, H, I, "mxfp4")
    inf, nan = np.inf, np.nan
    logits = np.array([[-inf, 1, -inf, -inf, -inf, -inf], [nan, nan, nan, 2, 1, 0.5],
                       [-inf] * 6, [nan] * 6, [inf, 0, inf, 5, 5, 5], [0, -0.0, 0, -0.0, 0, 0],
                       [-1e38, 1e38, 0, 3e38, -3e38, 0]], np.float32)
    # experts 0 and 2 hold NaN: only rows that weigh them may see it
    for e in (0, 2):
        for name in ("w13", "w2"):
            n = L.host[name][2]
            L.host[name][1][e * n // 16:(e + 1) * n // 16] = 255
    for rows in ([0], [0, 1, 2, 3], list(range(7)), list(range(7)) * 3):
        lg = logits[rows]
        x = R.bf16(np.random.default_rng(0).standard_normal((len(rows), H)))
        y, ids, w = bsq.moe_few_tokens(dev_rows(x), "mxfp4", *L.dev(), E, k,
                                       router_logits=torch.from_numpy(lg).cuda())
        torch.cuda.synchronize()
        wi, ww = R.route(lg.astype(np.float64), k, True)
        assert np.array_equal(ids.cpu().numpy(), wi)
        w = w.double().cpu().numpy()
        assert np.array_equal(w == 0, ww == 0) and np.allclose(w, ww, rtol=1e-5, atol=0)
        y = y.double().cpu().numpy()
        for t, r in enumerate(rows):
            sees = any(wi[t, j] in (0, 2) and ww[t, j] > 0 for j in range(k))
            assert sees == bool(np.isnan(y[t]).any()), (r, t)
            if not sees:
                want, bound = L.reference(x[t:t + 1], wi[t:t + 1], w[t:t + 1])
                assert np.all(np.abs(y[t] - want[0]) <= bound[0])
                assert ww[t].any() or np.all(y[t] == 0)


@pytest.mark.parametrize("T", [3, 30])
def test_entries_without_weight_and_equal_entries(bsq, T):  # noqa: F811
    """Weight 0, experts outside the layer and one expert twice for a token (its weights add)."""
    E, k, H, I = 5, 4, 256, 128
    L = Layer(2, E, H, I, "mxfp8")
    rng = np.random.default_rng(T)
    ids = rng.integers(-2, E + 2, (T, k)).astype(np.int32)
    ids[0] = [3, 3, 1, 3]
    ids[1] = [-1, 7, 100000, -2147483648]
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[rng.random((T, k)) < 0.2] = 0
    w[0] = [0, 0.5, 1, 0.25]
    x = R.bf16(rng.standard_normal((T, H)))
    y, _, _ = bsq.moe_few_tokens(dev_rows(x), "mxfp8", *L.dev(), E, k, topk_ids=i32(ids),
                                 topk_weights=torch.from_numpy(w).cuda())
    torch.cuda.synchronize()
    check(y, *L.reference(x, ids, w))
    assert torch.all(y[1] == 0)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("T", [1, 20])
def test_scale_bytes_at_the_ends(bsq, fmt, T):  # noqa: F811
    """E8M0 from 2^-127 to 2^20 in the weights: products exact, sums in range."""
    E, k, H, I = 3, 2, 256, 128
    L = Layer(3, E, H, I, fmt)
    rng = np.random.default_rng(3)
    for name in ("w13", "w2"):
        s = L.host[name][1]
        s[rng.random(s.shape) < 0.3] = 0
        s[rng.random(s.shape) < 0.1] = 1
        s[(rng.random(s.shape) < 0.1) & (s != 255)] = 135
    x = R.bf16(rng.standard_normal((T, H)))
    ids, w = given(5, T, E, k)
    y, _, _ = bsq.moe_few_tokens(dev_rows(x), fmt, *L.dev(), E, k, topk_ids=i32(ids),
                                 topk_weights=torch.from_numpy(w).cuda())
    torch.cuda.synchronize()
    check(y, *L.reference(x, ids, w))


def test_large_and_small_gates(bsq):  # noqa: F811
    """Gates from -3e4 to 3e4 and zeros: the SiLU neither overflows nor makes NaN."""
    E, k, H, I = 2, 1, 128, 128
    L = Layer(4, E, H, I, "mxfp4")
    x = R.bf16(np.random.default_rng(1).standard_normal((6, H)) * np.array([[1e-3], [1], [300], [3e3], [0], [1e-20]]))
    ids, w = given(1, 6, E, k)
    y, _, _ = bsq.moe_few_tokens(dev_rows(x), "mxfp4", *L.dev(), E, k, topk_ids=i32(ids),
                                 topk_weights=torch.from_numpy(w).cuda())
    torch.cuda.synchronize()
    check(y, *L.reference(x, ids, w))
    assert torch.all(y[4] == 0)


def test_strides_streams_and_same_bits(bsq):  # noqa: F811
    E, k, H, I = 12, 4, 256, 256
    L = Layer(5, E, H, I, "mxfp4")
    for T in (3, 40):
        x = R.bf16(np.random.default_rng(T).standard_normal((T, H)))
        ids, w = given(T, T, E, k)
        wide = torch.full((T, H + 24), 5.0, dtype=torch.bfloat16, device="cuda")
        wide[:, 8:H + 8] = dev_rows(x)
        out = torch.full((T + 1, H + 16), 3.0, dtype=torch.bfloat16, device="cuda")
        args = [wide[:, 8:H + 8], "mxfp4", *L.dev(), E, k]
        kw = dict(topk_ids=i32(ids), topk_weights=torch.from_numpy(w).cuda())
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        bsq.moe_few_tokens(*args, **kw, out=out[:T, :H], stream=side)
        torch.cuda.synchronize()
        check(out[:T, :H], *L.reference(x, ids, w))
        assert torch.all(out[T:] == 3) and torch.all(out[:, H:] == 3)
        for _ in range(4):
            assert torch.equal(bsq.moe_few_tokens(*args, **kw)[0], out[:T, :H])


def test_no_tokens_and_refusals(bsq):  # noqa: F811
    E, k, H, I = 4, 2, 128, 128
    L = Layer(6, E, H, I, "mxfp4")
    x = torch.zeros((0, H), dtype=torch.bfloat16, device="cuda")
    lg = torch.zeros((0, E), device="cuda")
    assert bsq.moe_few_tokens(x, "mxfp4", *L.dev(), E, k, router_logits=lg)[0].shape == (0, H)
    x = torch.zeros((2, H), dtype=torch.bfloat16, device="cuda")
    lg = torch.zeros((2, E), device="cuda")
    w = L.dev()
    for bad, kw in ((TypeError, dict(x=x.float())), (TypeError, dict(x=x.t())),
                    (bsq.BsqError, dict(fmt="nvfp4")), (bsq.BsqError, dict(fmt="mxfp8")),
                    (bsq.BsqError, dict(E=3)), (bsq.BsqError, dict(k=5)), (bsq.BsqError, dict(k=0)),
                    (bsq.BsqError, dict(router_logits=lg[:1])), (TypeError, dict(router_logits=lg.double())),
                    (bsq.BsqError, dict(router_logits=None)),
                    (bsq.BsqError, dict(out=torch.zeros((2, H + 128), dtype=torch.bfloat16, device="cuda"))),
                    (bsq.BsqError, dict(x=x.repeat(33, 1), router_logits=lg.repeat(33, 1)))):
        a = dict(dict(x=x, fmt="mxfp4", E=E, k=k, router_logits=lg, out=None), **kw)
        with pytest.raises(bad):
            bsq.moe_few_tokens(a["x"], a["fmt"], *w, a["E"], a["k"], router_logits=a["router_logits"],
                               out=a["out"])


@pytest.mark.parametrize("topk", [13, 1 << 31, 1 << 40, (1 << 63) - 1])
def test_far_topk_is_refused_before_memory_is_taken(bsq, topk):  # noqa: F811
    L = Layer(3, 12, 256, 128, "mxfp4")
    x, z = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, 12), device="cuda")
    with pytest.raises(bsq.BsqError, match="topk"):
        bsq.moe_few_tokens(x, "mxfp4", *L.dev(), 12, topk, router_logits=z)
