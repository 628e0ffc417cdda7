"""Routing and the grouped rows on the GPU: chosen experts and rows exactly, weights within the
reference's bounds; and the rows through the grouped quantizer and GEMM."""
import numpy as np
import pytest
import torch

import decoder_ref as R
from test_gpu_serving_kv import bsq, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def check(bsq, z, topk, dtype=torch.float32, bias=None, **kw):  # noqa: F811
    x = torch.tensor(z, device="cuda").to(dtype)
    b = None if bias is None else torch.tensor(bias, device="cuda").float()
    names = dict(groups="num_groups", keep="topk_groups", top="group_top")
    ids, w = bsq.moe_route(x, topk, bias=b, **{names.get(k, k): v for k, v in kw.items()})
    torch.cuda.synchronize()
    want, ww, bound = R.route(x.double().cpu().numpy(), topk, bias=None if b is None else b.double().cpu().numpy(),
                              **{**dict(score="softmax"), **kw})
    assert np.array_equal(ids.cpu().numpy(), want)
    off = np.abs(w.double().cpu().numpy() - ww)
    assert np.all(off <= bound), np.max(off / bound)
    return ids, w


SHAPES = [(1, 1, 1), (2, 8, 2), (5, 60, 6), (64, 128, 8), (7, 129, 16), (33, 256, 8), (3, 1000, 13), (4, 1024, 16)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sizes(bsq, T, E, k, score, bias, dtype):  # noqa: F811
    rng = np.random.default_rng(T + E + k)
    z, b = rng.standard_normal((T, E)) * 2, 0.1 * rng.standard_normal(E) if bias else None
    for renorm, factor in ((True, 1.0), (False, 2.5)):
        check(bsq, z, k, dtype, b, score=score, renormalize=renorm, factor=factor)


@pytest.mark.parametrize("E,groups,keep", [(256, 8, 4), (64, 64, 20), (12, 3, 1), (160, 8, 3), (1024, 2, 1),
                                           (1000, 40, 7), (6, 6, 6), (63, 9, 5)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_groups(bsq, E, groups, keep, top, score, bias):  # noqa: F811
    rng = np.random.default_rng(E + groups)
    z, b = rng.standard_normal((17, E)) * 2, 0.1 * rng.standard_normal(E) if bias else None
    k = min(8, E // groups * keep)
    check(bsq, z, k, bias=b, score=score, groups=groups, keep=keep, top=top, renormalize=top == 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 1), (4, 2)])
@pytest.mark.parametrize("bias", [False, True])
def test_equal_values_go_by_number(bsq, score, groups, top, bias):  # noqa: F811
    rng = np.random.default_rng(9)
    z = rng.integers(-1, 2, (40, 64)).astype(float)
    z[0] = 0.0
    z[1] = -0.0
    z[1, ::2] = 0.0
    b = rng.integers(0, 2, 64) * 0.5 if bias else None
    check(bsq, z, 10, bias=b, score=score, groups=groups, keep=max(1, groups // 2), top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_that_32_bits_cannot_tell_apart(bsq, score):  # noqa: F811
    """Biases that bring the scores of all experts to one value but for the rounding of the bias:
    the order of 64 bits."""
    rng = np.random.default_rng(3)
    z = rng.standard_normal(96).astype(np.float32).astype(float)
    s = 1 / (1 + np.exp(-z)) if score == "sigmoid" else np.exp(z) / np.exp(z).sum()
    b = (1.5 - s).astype(np.float32).astype(float)
    c = s + b
    assert np.unique(c.astype(np.float32)).size < 12 and np.unique(c).size == 96
    check(bsq, np.stack([z] * 3), 16, bias=b, score=score)
    check(bsq, np.stack([z] * 3), 8, bias=b, score=score, groups=8, keep=3, top=2)
    check(bsq, np.stack([z] * 3), 8, bias=b, score=score, groups=12, keep=5, top=1)
    # pairs of experts whose sums alone decide between groups
    z = np.repeat(rng.standard_normal((1, 32)), 4, 0).astype(np.float32).astype(float)
    z = z.reshape(4, 8, 4).transpose(0, 2, 1).reshape(4, 32)
    check(bsq, z, 4, score=score, groups=4, keep=2, top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("bias", [False, True])
def test_special_logits(bsq, score, renorm, bias):  # noqa: F811
    inf, nan = np.inf, np.nan
    rng = np.random.default_rng(8)
    z = rng.standard_normal((12, 16))
    z[0] = -inf
    z[1] = nan
    z[2, :13] = -inf
    z[3, ::2] = nan
    z[4, 3] = z[4, 11] = inf
    z[5] = 200 * z[5]
    z[6] = -300 + z[6]
    z[7] = 1e30 * np.sign(z[7])
    z[8, :8] = -1e4
    z[9] = [-3e38, 3e38] * 8
    z[10] = 30 + 0.01 * z[10]
    b = None
    if bias:
        b = 0.1 * rng.standard_normal(16)
        b[2], b[3], b[5], b[9] = -inf, nan, inf, -5.0
    for g in (dict(), dict(groups=4, keep=2), dict(groups=4, keep=2, top=2)):
        if score == "sigmoid" and bias is False and g.get("top") == 2:
            continue                 # sums of saturated scores: below, with a bias
        check(bsq, z, 4, bias=b, score=score, renormalize=renorm, **g)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,groups", [(16, 4), (160, 8), (512, 16)])
def test_sums_of_two_saturated_scores(bsq, E, groups, renorm):  # noqa: F811
    """Sigmoid scores that are 1 in 32 or in 64 bits, 0, or masked, without a bias: groups go by the
    sums in 64 bits, equal ones by their number, and the experts in them by their logits."""
    inf, nan = np.inf, np.nan
    rng = np.random.default_rng(E)
    z = rng.standard_normal((14, E))
    z[0] = 60 + 5 * z[0]                             # 1 in 64 bits: the first groups
    z[1] = 20 + 2 * z[1]                             # 1 in 32 bits, told apart in 64
    z[2] = 200 * z[2]
    z[3] = 1e30 * np.sign(z[3]) * (1 + rng.random(E))
    z[4, ::3] = inf
    z[5, ::2] = nan
    z[6, E // groups + 1:] = -inf                    # one group whole, the next with one expert
    z[7, rng.random(E) < 0.8] = -inf
    z[8] = -200 + 10 * z[8]                          # sums of 1e-87: 32 bits have none of them
    z[9] = -900 + z[9]                               # 0 in 64 bits too
    z[10] = np.where(np.arange(E) % 2, 50.0, -50.0) + z[10]
    z[11], z[12] = -inf, nan
    z[13, [1, E - 1]] = inf
    for keep in (1, 2, groups - 1):
        check(bsq, z, min(8, E // groups * keep), score="sigmoid", groups=groups, keep=keep, top=2, renormalize=renorm)


@pytest.mark.parametrize("E", [16, 200, 400])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinite_logits_that_are_not_chosen(bsq, E, renorm, dtype):  # noqa: F811
    """Under softmax they take the whole score all the same: where the chosen experts have none of
    it, their weights are 0."""
    inf, nan = np.inf, np.nan
    rng = np.random.default_rng(E)
    z, b = rng.standard_normal((6, E)), 0.1 * rng.standard_normal(E)
    b[[1, 5, 9]] = -inf, nan, -3.0
    z[0, 1] = z[1, 5] = z[2, 9] = inf
    z[3, [1, 5, 9]] = inf
    z[4, [1, 7]] = inf               # one of two is chosen
    x = torch.tensor(z, device="cuda").to(dtype)
    z, bf = x.double().cpu().numpy(), torch.tensor(b).float().double().numpy()
    for kw in (dict(), dict(groups=4, keep=3), dict(groups=4, keep=3, top=2)):
        want = R.route(z, 4, "softmax", bias=bf, renormalize=renorm, factor=1.5, **kw)
        s = np.isinf(z) / np.maximum(np.isinf(z).sum(1, keepdims=True), 1)
        s = np.take_along_axis(s, want[0], 1)[:5]
        total = s.sum(1, keepdims=True) if renorm else 1.0
        ids, w = bsq.moe_route(x, 4, bias=torch.tensor(b, device="cuda").float(), renormalize=renorm, factor=1.5,
                               **{dict(groups="num_groups", keep="topk_groups", top="group_top")[k]: v
                                  for k, v in kw.items()})
        torch.cuda.synchronize()
        assert np.array_equal(ids.cpu().numpy(), want[0])
        got = w.double().cpu().numpy()
        assert np.array_equal(got[:5], np.where(total > 0, 1.5 * s / np.maximum(total, 1e-9), 0.0))
        assert not got[:4].any() and got[4].any() and np.all(np.abs(got[5] - want[1][5]) <= want[2][5])
    # no bias: a group whose second best is -inf is not kept
    z = np.full((1, E), 0.5)
    z[0, :E // 4] = -inf
    z[0, 3] = inf
    ids, w = bsq.moe_route(torch.tensor(z, device="cuda").to(dtype), 4, num_groups=4, topk_groups=2, group_top=2,
                           renormalize=renorm)
    torch.cuda.synchronize()
    assert ids[0].tolist() == [E // 4 + i for i in range(4)] and not w.any()


def test_rows_of_a_larger_tensor(bsq):  # noqa: F811
    """A row stride, an odd offset of BF16 elements, outputs of the caller's."""
    rng = np.random.default_rng(2)
    big = torch.tensor(rng.standard_normal((9, 77)), device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        x = big.to(dtype)[:, 3:64]
        ids = torch.full((11, 5), -7, dtype=torch.int32, device="cuda")
        w = torch.full((11, 5), 7.0, device="cuda")
        r = bsq.moe_route(x, 5, topk_ids=ids, topk_weights=w)
        a = bsq.moe_route(x.contiguous(), 5)
        torch.cuda.synchronize()
        assert r[0] is ids and torch.equal(ids[:9], a[0]) and torch.equal(w[:9], a[1])
        assert bool((ids[9:] == -7).all()) and bool((w[9:] == 7).all())


def test_many_tokens(bsq):  # noqa: F811
    rng = np.random.default_rng(1)
    z = rng.standard_normal((1501, 64))
    check(bsq, z, 6, bias=0.1 * rng.standard_normal(64), score="sigmoid", groups=8, keep=3, top=2, factor=-1.5)
    ids, w = bsq.moe_route(torch.empty((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)


@pytest.mark.parametrize("E,k", [(5, 5), (16, 1), (17, 16), (64, 6), (65, 8), (128, 8), (129, 16), (200, 3), (256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_four_tokens_a_wave(bsq, E, k, score, renorm):  # noqa: F811
    """Many tokens without a bias: ties, masked experts and special logits among them."""
    rng = np.random.default_rng(E + k)
    z = rng.standard_normal((307 if E <= 64 else 4099 if E <= 128 else 8195, E)) * 2
    z[:200] = np.round(z[:200])
    z[200:220] *= 100
    z[220:240] -= 300
    z[240:260][rng.random((20, E)) < 0.7] = -np.inf
    z[260:280][rng.random((20, E)) < 0.5] = np.nan
    z[280:290][rng.random((10, E)) < 0.2] = np.inf
    z[290], z[291] = -np.inf, np.nan
    z[292, 0] = -0.0
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.tensor(z, device="cuda").to(dtype)
        few = [bsq.moe_route(t, k, score=score, renormalize=renorm, factor=1.5) for t in x.split(2000)]
        many = bsq.moe_route(x, k, score=score, renormalize=renorm, factor=1.5)
        torch.cuda.synchronize()
        assert torch.equal(many[0], torch.cat([f[0] for f in few]))
        assert torch.allclose(many[1], torch.cat([f[1] for f in few]), rtol=2e-6, atol=1e-37)
    check(bsq, z, k, score=score, renormalize=renorm, factor=1.5)
    x = torch.tensor(z, device="cuda").to(torch.bfloat16)
    wide = torch.full((len(z), E + 3), 1e9, device="cuda", dtype=torch.bfloat16)
    wide[:, 1:E + 1] = x
    for a, b in zip(bsq.moe_route(wide[:, 1:E + 1], k, score=score), bsq.moe_route(x, k, score=score)):
        assert torch.equal(a, b)


def test_route_agrees_with_moe_few_tokens(bsq):  # noqa: F811
    """Softmax routing chooses and weighs as moe_few_tokens does from the same logits."""
    from test_gpu_serving_moe import Layer

    rng = np.random.default_rng(4)
    L = Layer(9, 12, 256, 128, "mxfp4")
    x = torch.tensor(rng.standard_normal((9, 256)), device="cuda").to(torch.bfloat16)
    z = torch.tensor(rng.standard_normal((9, 12)), device="cuda").float()
    w = L.dev()
    for renorm in (True, False):
        y, ids, ws = bsq.moe_few_tokens(x, "mxfp4", *w, 12, 3, router_logits=z, renormalize=renorm)
        i2, w2 = bsq.moe_route(z, 3, renormalize=renorm)
        y2, _, _ = bsq.moe_few_tokens(x, "mxfp4", *w, 12, 3, topk_ids=i2, topk_weights=w2)
        torch.cuda.synchronize()
        assert torch.equal(ids, i2) and torch.allclose(ws, w2, rtol=1e-6, atol=0)
        assert torch.allclose(y.float(), y2.float(), rtol=2 ** -7, atol=1e-3)


# ------------------------------------------------------------------ grouped rows


def check_rows(bsq, ids, E, pad, **kw):  # noqa: F811
    got = bsq.moe_group_rows(i32(ids), E, pad=pad, **kw)
    torch.cuda.synchronize()
    want = R.group_rows(np.asarray(ids), E, pad)
    for name, g, w in zip(("row_offsets", "scales_offsets", "row_indices", "entry_rows"), got, want):
        assert np.array_equal(g.cpu().numpy(), w), name
    return got


@pytest.mark.parametrize("T,k", [(1, 1), (1, 16), (3, 2), (63, 1), (64, 8), (65, 7), (512, 8), (513, 8), (700, 12),
                                 (3000, 5)])
@pytest.mark.parametrize("E,pad", [(1, 16), (2, 1), (63, 128), (64, 7), (256, 128), (1023, 16), (1024, 65536)])
def test_group_rows(bsq, T, k, E, pad):  # noqa: F811
    rng = np.random.default_rng(T + k + E)
    check_rows(bsq, rng.integers(0, E, (T, k)), E, pad)
    check_rows(bsq, rng.integers(-2, E + 2, (T, k)), E, pad)


@pytest.mark.parametrize("T", [50, 2000])
def test_group_rows_of_uneven_choices(bsq, T):  # noqa: F811
    """Every entry one expert's; none anyone's; the same expert twice in a token; far numbers."""
    check_rows(bsq, np.full((T, 4), 5), 9, 128)
    check_rows(bsq, np.full((T, 4), -1), 9, 128)
    check_rows(bsq, np.full((T, 4), 2 ** 31 - 1), 1024, 128)
    check_rows(bsq, np.sort(np.random.default_rng(1).integers(0, 300, (T, 4)).reshape(-1)).reshape(T, 4), 300, 16)


def test_group_rows_of_many_tiles(bsq):  # noqa: F811
    rng = np.random.default_rng(5)
    check_rows(bsq, (rng.random((60000, 5)) ** 3 * 200).astype(int), 200, 128)
    # tiles of more entries than a wave keeps
    ids = torch.tensor(rng.integers(-1, 1024, (70001, 9)), dtype=torch.int32, device="cuda")
    rows, scales, index, entry = bsq.moe_group_rows(ids, 1024, pad=16)
    flat = ids.view(-1).long()
    key = torch.where(flat < 0, 1024, flat)
    order = torch.sort(key, stable=True)[1]
    counts = torch.bincount(key, minlength=1025)[:1024]
    n = int(counts.sum())
    assert torch.equal(rows[1:].long(), counts.cumsum(0)) and rows[0] == 0
    assert torch.equal(scales[1:].long(), ((counts + 15) // 16 * 16).cumsum(0)) and scales[0] == 0
    assert torch.equal(index[:n].long(), order[:n] // 9) and bool((index[n:] == -1).all())
    back = torch.full_like(flat, -1)
    back[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(entry.view(-1).long(), back)
    r = bsq.moe_group_rows(torch.empty((0, 3), dtype=torch.int32, device="cuda"), 70)
    torch.cuda.synchronize()
    assert not r[0].any() and not r[1].any() and r[0].numel() == 71 and r[2].numel() == 0


@pytest.mark.parametrize("E", [3, 130])
def test_group_rows_of_the_most_tiles(bsq, E):  # noqa: F811
    rng = np.random.default_rng(E)
    check_rows(bsq, rng.integers(-1, E + 1, (300001, 4)), E, 16)


def test_group_rows_outputs_of_the_callers(bsq):  # noqa: F811
    ids = np.random.default_rng(6).integers(0, 8, (900, 6))
    want = check_rows(bsq, ids, 8, 16)
    ro = torch.zeros(9, dtype=torch.uint32, device="cuda")
    ri = torch.full((6000,), 9, dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    got = bsq.moe_group_rows(i32(ids), 8, pad=16, row_offsets=ro, row_indices=ri, workspace=ws)
    torch.cuda.synchronize()
    assert got[0] is ro and torch.equal(ro.view(torch.int32), want[0])
    assert torch.equal(ri[:5400], want[2]) and bool((ri[5400:] == 9).all())


@pytest.mark.parametrize("T", [40, 900])
def test_rows_through_the_grouped_calls(bsq, T):  # noqa: F811
    """Route, group, quantize with the gather, multiply, and add up by entry_rows: equal to each
    entry's own product."""
    g = torch.Generator(device="cuda").manual_seed(T)
    E, k, H, N = 10, 3, 256, 128
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((E * N, H), generator=g, device="cuda").to(torch.bfloat16)
    z = torch.randn((T, E), generator=g, device="cuda")
    ids, weights = bsq.moe_route(z, k, score="sigmoid")
    rows, scales, index, entry = bsq.moe_group_rows(ids, E, pad=128)
    most = T * k + E * 127
    most -= most % 128
    experts = torch.arange(E, dtype=torch.int32, device="cuda")
    wc, ws = bsq.quantize_block_scaled(w, "mxfp8", scale_layout=bsq.SCALES_MFMA16)
    xc, xs = bsq.grouped_quantize_block_scaled(x, "mxfp8", rows, scales, experts, None, T * k, most,
                                               row_indices=index, scale_layout=bsq.SCALES_MFMA16)
    c = bsq.grouped_block_scaled_matmul_mfma(xc, xs, rows, scales, experts, T * k, most, wc, ws, E,
                                             "mxfp8", H)
    y = (c[entry.long()] * weights[..., None]).sum(1)
    dq, ds = bsq.quantize_block_scaled(x, "mxfp8")
    a = bsq.dequantize_block_scaled(dq, ds, "mxfp8", H).double()
    dq, ds = bsq.quantize_block_scaled(w, "mxfp8")
    b = bsq.dequantize_block_scaled(dq, ds, "mxfp8", H).double().view(E, N, H)
    torch.cuda.synchronize()
    want, size = torch.zeros((2, T, N), dtype=torch.float64, device="cuda")
    for j in range(k):
        for e in range(E):
            t = (ids[:, j] == e).nonzero()[:, 0]
            f = weights[t, j, None].double()
            want[t] += f * (a[t] @ b[e].t().contiguous())
            size[t] += f * (a[t].abs() @ b[e].abs().t().contiguous())
    # two 128-element steps, each off by 2^-12 of its largest product at most, and fp32 sums
    assert bool(((y - want).abs() <= size * 2.0 ** -11).all())


def test_refusals_of_the_binding(bsq):  # noqa: F811
    z, ids = torch.zeros((4, 16), device="cuda"), i32([[1, 2]] * 4)
    b = torch.zeros(16, device="cuda")
    for err, kw in [(TypeError, dict(logits=z.half())), (TypeError, dict(logits=z.cpu())),
                    (TypeError, dict(logits=z[0])), (TypeError, dict(logits=z.t())),
                    (TypeError, dict(bias=b.double())), (TypeError, dict(topk=1.5)),
                    (TypeError, dict(topk_ids=ids.long())), (bsq.BsqError, dict(topk_ids=ids[:3])),
                    (bsq.BsqError, dict(topk_weights=z[:, :3].contiguous())), (bsq.BsqError, dict(topk=0)),
                    (bsq.BsqError, dict(topk=17)), (bsq.BsqError, dict(bias=b[:8])),
                    (bsq.BsqError, dict(num_groups=3)), (bsq.BsqError, dict(num_groups=8, topk_groups=9)),
                    (bsq.BsqError, dict(num_groups=16, topk_groups=1)), (bsq.BsqError, dict(group_top=3)),
                    (bsq.BsqError, dict(factor=float("nan"))), (bsq.BsqError, dict(score="tanh"))]:
        args = dict(logits=z, topk=2)
        args.update(kw)
        with pytest.raises(err):
            bsq.moe_route(**args)
    for err, kw in [(TypeError, dict(topk_ids=ids.long())), (TypeError, dict(topk_ids=ids[:, :1])),
                    (TypeError, dict(topk_ids=ids[0])), (bsq.BsqError, dict(num_experts=0)),
                    (bsq.BsqError, dict(num_experts=1025)), (bsq.BsqError, dict(pad=0)),
                    (bsq.BsqError, dict(pad=65537)), (bsq.BsqError, dict(topk_ids=ids[:, :0])),
                    (bsq.BsqError, dict(row_offsets=ids[:, 0].contiguous())),
                    (bsq.BsqError, dict(row_indices=ids[:2].reshape(-1))), (TypeError, dict(entry_rows=z))]:
        args = dict(topk_ids=ids, num_experts=4)
        args.update(kw)
        with pytest.raises(err):
            bsq.moe_group_rows(**args)


@pytest.mark.parametrize("topk", [17, 1025, 1 << 31, 1 << 40, (1 << 63) - 1])
@pytest.mark.parametrize("T", [0, 4])
def test_far_topk_is_refused_before_memory_is_taken(bsq, topk, T):  # noqa: F811
    z = torch.zeros((T, 16), device="cuda")
    with pytest.raises(bsq.BsqError, match="topk"):
        bsq.moe_route(z, topk)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("step", [2.0 ** -25, 2.0 ** -22, 2.0 ** -19, 2.0 ** -16, 2.0 ** -13])
@pytest.mark.parametrize("groups", [1, 8])
def test_gaps_of_every_size(bsq, score, step, groups):  # noqa: F811
    """Scores plus biases that lie `step` apart, or equal, in random order: sizes where 32 bits
    tell them apart, where they cannot, and between."""
    rng = np.random.default_rng(int(1 / step) % 1000 + groups)
    E = 64
    z = np.float32(rng.standard_normal((20, E)) * 1.5).astype(float)
    s = 1 / (1 + np.exp(-z)) if score == "sigmoid" else np.exp(z) / np.exp(z).sum(1, keepdims=True)
    for t in range(4):
        place = rng.permutation(E) // (2 if t % 2 else 1)
        b = np.float32(0.7 + place * step - s[t]).astype(float)
        check(bsq, z[t:t + 1], 8, bias=b, score=score, groups=groups, keep=max(1, groups // 2), top=2)
        # the same biases for other tokens: ordinary gaps beside
        check(bsq, z, 8, bias=b, score=score, groups=groups, keep=max(1, groups // 2), top=1)


def test_few_experts_left(bsq):  # noqa: F811
    """As many experts with a finite choice as are asked for, one more and one less."""
    rng = np.random.default_rng(0)
    z = rng.standard_normal((3, 32))
    for left in (3, 4, 5):
        x = z.copy()
        x[:, left:] = -np.inf
        for score in ("softmax", "sigmoid"):
            check(bsq, x, 4, bias=0.1 * rng.standard_normal(32), score=score)
            check(bsq, x, 4, bias=0.1 * rng.standard_normal(32), score=score, groups=4, keep=2, top=2)
