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
