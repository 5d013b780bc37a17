"""A 4-bit tensor decodes with the tensorwise scale that its codes were made
with, also after its ScalingState has moved on."""
import numpy as np
import pytest
import torch

import quantised_gemm_gb300 as q
from helpers import assert_within_bound, bf16_to_f64, to_dev_bf16
from oracle import fp4 as o4

pytestmark = pytest.mark.gpu


def values(t):
    return q.fp4_dequantise(t, torch.empty((t.rows, t.cols), device="cuda"))


def bits_of(rows, cols, seed, std=1.0):
    x = (np.random.default_rng(seed).normal(size=(rows, cols)) * std).astype(np.float32)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    return bits, (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def exact(x, scale):
    """What x ([rows, cols]) stands for at the tensorwise scale (S, inv)."""
    codes, sc = o4.quantise(np.ascontiguousarray(x), o4.NVFP4, scale[0])
    return o4.values(codes, sc, o4.NVFP4, x.shape[1], scale[1])


@pytest.mark.parametrize("rows,cols", [(1, 16), (40, 100), (700, 1100)])
def test_two_tensors_of_one_state(rows, cols):
    ws, st = q.Workspace(), q.ScalingState(q.E4M3, q.DYNAMIC, amax_algo=q.AMAX_AUTO)
    first = q.Fp4Tensor(rows, cols, state=st), q.Fp4Tensor(cols, rows, state=st)
    second = q.Fp4Tensor(rows, cols, state=st), q.Fp4Tensor(cols, rows, state=st)
    (xb, x), (yb, y) = bits_of(rows, cols, 1), bits_of(rows, cols, 2, 30.0)
    q.fp4_quantise(to_dev_bf16(xb), *first, ws)
    q.fp4_quantise(to_dev_bf16(yb), *second, ws)
    for (t, tt), v in ((first, x), (second, y)):
        s = o4.tensor_scale(np.abs(v).max())
        for got, m in ((t, v), (tt, v.T)):
            want = exact(m, s)
            # fp32 values: the two roundings of their products.
            assert np.all(np.abs(values(got).cpu().numpy() - want) <= 2.0 ** -23 * np.abs(want))
            assert float(got.inv_scale) == s[1]


@pytest.mark.parametrize("M,N", [(3, 640), (200, 640)])
def test_delayed_tensor_after_the_next_scale(M, N):
    """M = 3: quantised in the product's launch."""
    K = 512
    ws, st = q.Workspace(), q.ScalingState(q.E4M3, q.DELAYED, history_len=1)
    w4 = q.Fp4Tensor(N, K)
    q.fp4_quantise(to_dev_bf16(bits_of(N, K, 3)[0]), w4, None, ws)
    scale = None
    for step in range(3):
        x4 = q.Fp4Tensor(M, K, state=st)
        xb, x = bits_of(M, K, 10 + step, 8.0 ** step)
        scale = scale or o4.tensor_scale(np.abs(x).max())   # the first cast takes its own
        y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        q.fp4_linear(to_dev_bf16(xb), x4, w4, y, ws)
        before = values(x4)
        q.scale(st)
        assert float(x4.inv_scale) == scale[1]
        want = exact(x, scale)
        scale = o4.tensor_scale(np.abs(x).max())
        assert float(st.inv_scale) == scale[1]
        assert torch.equal(values(x4), before)
        assert np.all(np.abs(before.cpu().numpy() - want) <= 2.0 ** -23 * np.abs(want))
        assert torch.equal(q.fp4_gemm(x4, w4, torch.empty_like(y), ws), y)


@pytest.mark.parametrize("M,K,N", [(48, 160, 96), (300, 512, 384)])
def test_delayed_backward_after_sync(M, K, N):
    lin = q.Fp4Linear(M, K, N, scaling="delayed", history_len=1)
    (db, dy) = bits_of(M, N, 3, 1e-3)
    sx = sw = None
    for step in range(3):
        (xb, x), (wb, w) = bits_of(M, K, 20 + step, 5.0 ** step), bits_of(N, K, 30 + step, 0.05 * 3.0 ** step)
        sx, sw = sx or o4.tensor_scale(np.abs(x).max()), sw or o4.tensor_scale(np.abs(w).max())
        lin.forward(to_dev_bf16(xb), to_dev_bf16(wb))
        lin.sync_scales()
        dx, dw = lin.backward(to_dev_bf16(db))
        q.check(lin.ws)
        # dY has no amax on record before its first cast, and the same one after it.
        sd = o4.tensor_scale(np.abs(dy).max())
        d4, d4t, w4t, x4t = exact(dy, sd), exact(dy.T, sd), exact(w.T, sw), exact(x.T, sx)
        for got, a, b, what in ((dx, d4, w4t, "dX"), (dw, d4t, x4t, "dW")):
            assert_within_bound(bf16_to_f64(got), a @ b.T, np.abs(a) @ np.abs(b).T, what)
        sx, sw = o4.tensor_scale(np.abs(x).max()), o4.tensor_scale(np.abs(w).max())


def test_empty_tensor_has_its_states_scale():
    t = q.Fp4Tensor(0, 64)
    q.fp4_quantise(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), t, None, q.Workspace())
    assert torch.equal(t.inv_scale, t.state.inv_scale) and float(t.inv_scale) == o4.tensor_scale(0.0)[1]


@pytest.mark.parametrize("fmt", [q.NVFP4, q.MXFP4], ids=["nv", "mx"])
def test_backward_needs_a_forward(fmt):
    lin = q.Fp4Linear(16, 32, 48, fmt=fmt)
    x, w, dy = (torch.ones(s, dtype=torch.bfloat16, device="cuda") for s in ((16, 32), (48, 32), (16, 48)))
    with pytest.raises(ValueError):
        lin.backward(dy)
    lin.forward(x, w)
    dx, dw = lin.backward(dy)
    assert (dx == 48).all() and (dw == 16).all()


@pytest.mark.parametrize("fmt,scaling", [(q.NVFP4, "dynamic"), (q.NVFP4, "delayed"), (q.MXFP4, "dynamic")])
@pytest.mark.parametrize("M,K,N", [(0, 64, 48), (5, 0, 48), (5, 64, 0), (0, 0, 0)])
def test_empty_linear(M, K, N, fmt, scaling):
    lin = q.Fp4Linear(M, K, N, fmt=fmt, scaling=scaling)
    x, w, dy = (torch.ones(s, dtype=torch.bfloat16, device="cuda") for s in ((M, K), (N, K), (M, N)))
    for _ in range(2):
        for t in (lin.y, lin.dx, lin.dw):
            t.fill_(3.0)
        y = lin.forward(x, w)
        dx, dw = lin.backward(dy)
        lin.sync_scales()
        q.check(lin.ws)
        assert (y == 0).all() and (dx == 0).all() and (dw == 0).all()
    for st in (lin.sx, lin.sw):   # (an empty dX and dW leave dY alone)
        assert st is None or st.needs_init == 0
