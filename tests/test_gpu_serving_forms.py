"""The forms of the serving kernels that calls at serving sizes take, at sizes that the 64-bit
reference can follow: attention with four waves a workgroup, the experts' down products as a walk
over several experts, and inputs that are not finite."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_serving_kv import attend, bsq, check, dev_rows, i32, make  # noqa: F401
from test_gpu_serving_moe import Layer, check as close

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,group,seqs", [(1, 1, 70), (1, 4, 66), (5, 4, 34), (16, 4, 17)])
@pytest.mark.parametrize("window,max_kv", [(0, 0), (90, 0), (0, 6400)])
def test_four_waves_a_workgroup(bsq, D, rows, group, seqs, window, max_kv):  # noqa: F811
    """More than 512 workgroups: one block of 16 columns (whose pages no other workgroup reads), two
    and four; with a loose bound on the lengths the pages are split as well.  NaN scales among
    them."""
    heads = 8
    assert seqs * heads * -(-rows * group // 16) > 512
    rng = np.random.default_rng(seqs + D)
    lens = [int(n) for n in rng.integers(rows, 150, seqs)]
    n = [int(x) for x in rng.integers(max(1, rows // 2), rows + 1, seqs)]
    n[3] = rows
    if max_kv:
        lens[:2] = [2500, 2300]
        assert bsq.serving_lib().kv_cache_attention_workspace(
            heads, D, heads * group, seqs, sum(n), rows, max_kv, window) > 0
    c, q, off, table = make(D + rows, lens, n, heads, heads * group, D)
    c.ks[table[1][0], 2] = 255
    c.vs[table[5][0], 7] = 255
    c.ks[table[9][R.pages_of(lens[9]) - 1], 0] = 255
    check(bsq, c, q, off, lens, table, D ** -0.5, window, max_q=rows, max_kv=max_kv or max(lens))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,lens", [(1, [90, 40, 70]), (5, [4000, 64, 70]), (100, [150, 130, 140])])
def test_queries_that_are_not_finite(bsq, D, rows, lens):  # noqa: F811
    """A NaN or an infinity of q makes NaN of its own row and head."""
    c, q, off, table = make(D + rows, lens, [rows] * 3, 2, 8, D)
    c.k[(c.k & 0x7F) == 0] |= 8                              # an infinity times 0 is tested by NaN
    q[0, 1, 3] = np.nan
    q[rows, 6, D - 1] = np.inf
    q[3 * rows - 1, 0, 9] = -np.inf
    with np.errstate(invalid="ignore"):
        out = check(bsq, c, q, off, lens, table, D ** -0.5)
    bad = np.isnan(out).all(-1)
    assert bad.sum() == 3 and np.isnan(out).any(-1).sum() == 3
    assert bad[0, 1] and bad[rows, 6] and bad[3 * rows - 1, 0]


# ------------------------------------------------------------------ experts


@pytest.mark.parametrize("fmt,H,I,E,skew", [
    ("mxfp4", 8192, 128, 20, False), ("mxfp4", 8192, 128, 20, True), ("mxfp8", 8192, 128, 20, False),
    ("mxfp8", 8192, 128, 20, True), ("mxfp4", 8192, 384, 18, True), ("mxfp4", 15360, 640, 10, False),
    ("mxfp8", 8192, 640, 18, True)])
def test_down_products_over_several_experts(bsq, fmt, H, I, E, skew):  # noqa: F811
    """More experts in use than a column tile has workgroups (512 over the tiles of 256 columns):
    each walks on to another expert, over whole and partial steps; with one expert of every token
    it has more than two blocks of 16 entries."""
    T, k = 40, 2
    assert E > 512 // (-(-H // 256))
    L = Layer(H + I, E, H, I, fmt)
    rng = np.random.default_rng(I)
    x = R.bf16(rng.standard_normal((T, H)))
    if skew:
        ids = np.stack([np.full(T, E - 2), np.where(np.arange(T) % (E - 1) == E - 2, E - 1, np.arange(T) % (E - 1))], 1)
        ids[:, 1] = np.where(ids[:, 1] == E - 2, 0, ids[:, 1])
    else:
        ids = np.stack([np.arange(T) % E, (np.arange(T) * 3 + 1) % E], 1)
    assert len(np.unique(ids)) > 512 // (-(-H // 256)) and np.all(ids[:, 0] != ids[:, 1])
    w = rng.random((T, k)).astype(np.float32) + 0.1
    y, _, _ = bsq.moe_few_tokens(dev_rows(x), fmt, *L.dev(), E, k, topk_ids=i32(ids),
                                 topk_weights=torch.from_numpy(w).cuda())
    torch.cuda.synchronize()
    close(y, *L.reference(x, ids, w))


@pytest.mark.parametrize("T", [1, 3, 16, 30])
def test_tokens_that_are_not_finite(bsq, T):  # noqa: F811
    """A NaN or an infinity of x makes NaN of its own token, also where tokens share experts."""
    E, k, H, I = 3, 2, 256, 128
    L = Layer(T, E, H, I, "mxfp4")
    rng = np.random.default_rng(T)
    x = R.bf16(rng.standard_normal((T, H)))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    w = rng.random((T, k)).astype(np.float32) + 0.1
    fine = np.ones(T, bool)
    for t, v in ((0, np.nan), (T - 1, np.inf)):
        bad = x.copy()
        bad[t, 7] = v
        y, _, _ = bsq.moe_few_tokens(dev_rows(bad), "mxfp4", *L.dev(), E, k, topk_ids=i32(ids),
                                     topk_weights=torch.from_numpy(w).cuda())
        torch.cuda.synchronize()
        y = y.double().cpu().numpy()
        want, bound = L.reference(x, ids, w)
        fine[:] = True
        fine[t] = False
        assert np.isnan(y[t]).all()
        assert np.all(np.abs(y - want)[fine] <= bound[fine])
