"""Edges of the serving operators: pages without a number in their scale beside far smaller ones,
numbers at the ends of their range."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_serving_kv import bsq, check, dev_rows, i32, make  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention


@pytest.mark.parametrize("D,heads", [(64, 1), (128, 2), (256, 1)])
@pytest.mark.parametrize("vs", [7, 27, 60])
@pytest.mark.parametrize("rows,L,window", [(2, 664, 600), (130, 330, 200)])
def test_nan_page_that_a_row_does_not_see(bsq, D, heads, vs, rows, L, window):  # noqa: F811
    """The first page has the NaN scale and the window of the later rows starts past it; V's
    other scales are 2^-120 to 2^-67: those rows keep every bit of V.  664 tokens: the wave that
    meets the NaN page has another page after it."""
    c, q, off, table = make(D + vs, [L], [rows], heads, 2 * heads, D)
    c.vs[:] = vs
    c.vs[table[0][0]] = 255
    out = check(bsq, c, q, off, [L], table, D ** -0.5, window)
    assert np.isnan(out).any() and np.isfinite(out).any()


# ------------------------------------------------------------------ experts


@pytest.mark.parametrize("T", [1, 3, 20])
def test_hidden_values_past_the_bf16_range(bsq, T):  # noqa: F811
    """A gated value between the largest BF16 number and the largest fp32 one stays that number,
    and one past fp32 is infinite, not NaN."""
    from test_gpu_serving_moe import Layer, check as close

    E, H, I = 2, 128, 128
    L = Layer(0, E, H, I, "mxfp8")
    for name, n, k in (("w13", 2 * I, H), ("w2", H, I)):
        codes, scales = L.host[name][:2]
        codes[:] = 0
        scales[:] = 127
    one = int(R.to_e4m3(1.0))
    codes, scales = L.host["w13"][:2]
    # W1 row: 2^64 x0; W3 row: 2^64 (x0 + x1)
    for e in range(E):
        codes[e * 2 * I:e * 2 * I + 2 * I, 0] = one
        codes[e * 2 * I + I:e * 2 * I + 2 * I, 1] = one
    scales[:] = 127 + 64
    codes, scales = L.host["w2"][:2]
    codes[:] = one
    scales[:] = 127 - 100
    x = np.zeros((T, H))
    x[:, 0] = 1.0
    x[:, 1] = -2.0 ** -11                                    # h = 2^128 - 2^117, BF16 ends at 2^128 - 2^120
    ids, w = np.zeros((T, 1), np.int32), np.full((T, 1), 0.5, np.float32)

    def run():
        return bsq.moe_few_tokens(dev_rows(x), "mxfp8", *L.dev(), E, 1, topk_ids=i32(ids),
                                  topk_weights=torch.from_numpy(w).cuda())[0]
    y = run()
    torch.cuda.synchronize()
    close(y, *L.reference(x, ids, w))
    assert abs(float(y[0, 0]) / (2.0 ** 34 * (1 - 2.0 ** -11)) - 1) <= 2.0 ** -8
    x[:, 1] = 1.0                                            # h = 2^129
    y = run()
    torch.cuda.synchronize()
    assert torch.all(y == np.inf)
