"""Norm and rotation of queries and keys on the GPU against the 64-bit reference."""
import numpy as np
import pytest
import torch

import decoder_ref as R
from test_gpu_serving_kv import bsq, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def inputs(rows, hq, hkv, D, rot, dtype, far=5000, seed=0):
    """q, k, v as slices of one projection, positions, inv_freq."""
    rng = np.random.default_rng(seed + rows + hq + D + rot)
    x = rng.standard_normal((rows, hq + 2 * hkv, D)) * np.exp2(rng.integers(-3, 4, (rows, 1, 1)))
    x = torch.tensor(x, device="cuda").to(dtype)
    f = 10000.0 ** (-2 * np.arange(rot // 2) / max(rot, 1))
    return (*x.split([hq, hkv, hkv], 1), rng.integers(0, far, rows), f, 1 + 0.2 * rng.standard_normal((2, D)))


def check(bsq, q, k, v, pos, f, w, eps=1e-6, interleaved=False, **kw):  # noqa: F811
    wd = [None, None] if w is None else [torch.tensor(x, device="cuda").float() for x in w]
    got = bsq.qk_norm_rope(q, k, i32(pos), torch.tensor(f, device="cuda"), v=v, q_weight=wd[0],
                           k_weight=wd[1], eps=eps, interleaved=interleaved, **kw)
    torch.cuda.synchronize()
    for g, x, x_w in zip(got, (q, k), wd):
        want, bound = R.norm_rope(x.double().cpu().numpy(), None if x_w is None else x_w.double().cpu().numpy(),
                                  float(np.float32(eps)), np.asarray(pos), np.asarray(f), interleaved)
        g = g.double().cpu().numpy()
        assert np.array_equal(np.isnan(g), np.isnan(want))
        ok = ~np.isnan(want)
        assert np.all(np.abs(g - want)[ok] <= bound[ok]), np.max((np.abs(g - want) / bound)[ok])
    if v is None:
        assert got[2] is None
    else:
        assert torch.equal(got[2], v.to(torch.bfloat16))
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (256, 256), (128, 32), (256, 64), (64, 16),
                                   (96, 96), (80, 48), (8, 0), (16, 16), (200, 192), (248, 0), (136, 112)])
def test_widths(bsq, D, rot, interleaved, dtype):  # noqa: F811
    q, k, v, pos, f, w = inputs(5, 7, 3, D, rot, dtype)
    check(bsq, q, k, v, pos, f, w, interleaved=interleaved)
    check(bsq, q, k, None, pos, f, None, interleaved=interleaved)


@pytest.mark.parametrize("rows", [1, 2, 63, 700])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (32, 8), (5, 5), (17, 1)])
def test_rows_and_heads(bsq, rows, hq, hkv):  # noqa: F811
    q, k, v, pos, f, w = inputs(rows, hq, hkv, 128, 128, torch.float32)
    check(bsq, q, k, v, pos, f, w)


def test_many_rows_take_several_heads_a_wave(bsq):  # noqa: F811
    q, k, v, pos, f, w = inputs(3001, 9, 2, 64, 64, torch.bfloat16)
    check(bsq, q, k, v, pos, f, w)


def test_one_weight_alone(bsq):  # noqa: F811
    q, k, _, pos, f, w = inputs(9, 4, 2, 64, 32, torch.bfloat16)
    qw = torch.tensor(w[0], device="cuda").float()
    a = bsq.qk_norm_rope(q, k, i32(pos), torch.tensor(f, device="cuda"), q_weight=qw)
    b = check(bsq, q, k, None, pos, f, None)
    c = check(bsq, q, k, None, pos, f, w)
    torch.cuda.synchronize()
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("pos", [[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 131072, 1 << 24, 1000003]])
def test_far_and_negative_positions(bsq, pos):  # noqa: F811
    q, k, v, _, f, w = inputs(len(pos), 4, 2, 128, 128, torch.float32)
    check(bsq, q, k, v, pos, f, w)


def test_frequencies_of_quarter_turns(bsq):  # noqa: F811
    """Angles at the borders of the reduction: multiples of an eighth of a turn."""
    f = np.arange(8) * np.pi / 4
    q, k, v, pos, _, w = inputs(33, 2, 2, 16, 16, torch.float32, far=100)
    check(bsq, q, k, v, pos, f, w)


def test_sizes_of_values(bsq):  # noqa: F811
    """Heads of zeros, of tiny and of large numbers; NaN and Inf stay in their head."""
    q, k, v, pos, f, w = inputs(8, 4, 2, 64, 64, torch.float32)
    q, k = q.clone(), k.clone()
    q[0] = 0
    q[1] *= 2.0 ** -40
    q[2] *= 2.0 ** 50
    k[3] *= 2.0 ** -60
    check(bsq, q, k, v, pos, f, w)
    check(bsq, q[1:2], k[1:2], v[1:2], pos[1:2], f, w, eps=0.0)
    check(bsq, q[3:4], k[3:4], v[3:4], pos[3:4], f, w, eps=0.0)
    q[4, 2, 5] = float("nan")
    q[5, 1, 63] = float("inf")
    got = bsq.qk_norm_rope(q, k, i32(pos), torch.tensor(f, device="cuda"),
                           q_weight=torch.ones(64, device="cuda"))[0]
    torch.cuda.synchronize()
    bad = got.isnan().any(-1).cpu()
    want = torch.zeros_like(bad)
    want[4, 2] = want[5, 1] = True
    assert torch.equal(bad, want)


def test_in_place_and_outputs_of_the_callers(bsq):  # noqa: F811
    q, k, v, pos, f, w = inputs(70, 8, 2, 128, 128, torch.bfloat16)
    want = check(bsq, q, k, None, pos, f, w)
    qkv = torch.cat([q, k, v], 1)
    a, b, c = qkv.split([8, 2, 2], 1)
    fd, wd = torch.tensor(f, device="cuda"), [torch.tensor(x, device="cuda").float() for x in w]
    r = bsq.qk_norm_rope(a, b, i32(pos), fd, q_weight=wd[0], k_weight=wd[1], q_out=a, k_out=b)
    torch.cuda.synchronize()
    assert r[0] is a and torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, v)
    big = torch.full((75, 12, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    bsq.qk_norm_rope(q, k, i32(pos), fd, v=v, q_weight=wd[0], k_weight=wd[1], q_out=big[:, :8],
                     k_out=big[:, 8:10], v_out=big[:, 10:])
    torch.cuda.synchronize()
    assert torch.equal(big[:70, :8], want[0]) and torch.equal(big[:70, 8:10], want[1])
    assert torch.equal(big[:70, 10:], v) and bool((big[70:] == 7).all())


def test_no_rows(bsq):  # noqa: F811
    q, k, v, pos, f, w = inputs(3, 2, 1, 64, 64, torch.bfloat16)
    r = bsq.qk_norm_rope(q[:0], k[:0], i32(pos[:0]), torch.tensor(f, device="cuda"), v=v[:0])
    assert [tuple(t.shape) for t in r] == [(0, 2, 64), (0, 1, 64), (0, 1, 64)]


def test_rows_past_32_bits(bsq):  # noqa: F811
    """Row strides whose products pass 2^32 elements: the last row of 2^17 at a stride of 2^15 + 8."""
    rows, ld = 1 << 17, (1 << 15) + 8
    x = torch.zeros(((rows - 1) * ld + 256,), dtype=torch.bfloat16, device="cuda")
    q = x.as_strided((rows, 2, 64), (ld, 64, 1))
    k = x.as_strided((rows, 2, 64), (ld, 64, 1), 128)
    g = torch.Generator(device="cuda").manual_seed(1)
    part = torch.randn((2, 4, 64), generator=g, device="cuda").to(torch.bfloat16)
    q[-2:], k[-2:] = part[:, :2], part[:, 2:]
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    f = torch.tensor(10000.0 ** (-np.arange(32) / 32), device="cuda")
    a, b, _ = bsq.qk_norm_rope(q, k, pos, f)
    c, d, _ = bsq.qk_norm_rope(part[:, :2], part[:, 2:], pos[-2:], f)
    torch.cuda.synchronize()
    assert torch.equal(a[-2:], c) and torch.equal(b[-2:], d) and not bool(a[:-2].any())


def test_refusals_of_the_binding(bsq):  # noqa: F811
    q, k, v, pos, f, w = inputs(4, 2, 1, 64, 64, torch.bfloat16)
    p, fd, w1 = i32(pos), torch.tensor(f, device="cuda"), torch.ones(64, device="cuda")
    for err, kw in [(TypeError, dict(q=q.float())), (TypeError, dict(q=q.half(), k=k.half())),
                    (TypeError, dict(positions=p.long())), (TypeError, dict(inv_freq=fd.float())),
                    (TypeError, dict(q_weight=w1.double())), (TypeError, dict(q=q.cpu())),
                    (TypeError, dict(q_out=q.float())), (TypeError, dict(q=q.transpose(1, 2))),
                    (TypeError, dict(eps="a")), (bsq.BsqError, dict(positions=p[:3])),
                    (bsq.BsqError, dict(q_weight=w1[:32])), (bsq.BsqError, dict(k=k[:3])),
                    (bsq.BsqError, dict(k=k[..., :32].contiguous())), (bsq.BsqError, dict(v=q)),
                    (bsq.BsqError, dict(inv_freq=fd[:7])), (bsq.BsqError, dict(inv_freq=fd.repeat(2))),
                    (bsq.BsqError, dict(q_out=q[:3])), (bsq.BsqError, dict(v_out=torch.empty_like(k))),
                    (bsq.BsqError, dict(eps=-1.0)), (bsq.BsqError, dict(eps=float("nan"))),
                    (bsq.BsqError, dict(q=torch.zeros(600, dtype=q.dtype, device="cuda")[4:516].view(4, 2, 64)))]:
        args = dict(q=q, k=k, positions=p, inv_freq=fd)
        args.update(kw)
        with pytest.raises(err):
            bsq.qk_norm_rope(**args)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_inputs_past_the_caches_size(bsq, dtype, interleaved):  # noqa: F811
    """More bytes than the memory-side cache holds are read another way: the same bits as in parts."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, cut = 12000, 7000
    q = torch.randn((rows, 32, 128), generator=g, device="cuda").to(dtype)
    k = torch.randn((rows, 12, 128), generator=g, device="cuda").to(dtype)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    f, w = torch.tensor(1000.0 ** (-np.arange(64) / 64), device="cuda"), torch.ones(128, device="cuda")
    a = bsq.qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w, interleaved=interleaved)
    for lo, hi in ((0, cut), (cut, rows)):
        b = bsq.qk_norm_rope(q[lo:hi], k[lo:hi], pos[lo:hi], f, q_weight=w, k_weight=w, interleaved=interleaved)
        torch.cuda.synchronize()
        assert torch.equal(a[0][lo:hi], b[0]) and torch.equal(a[1][lo:hi], b[1])
