"""Layer norm and its backward pass on the GPU against the formulas in 64 bits.

Bounds.  A sum of n fp32 terms in any order is off by at most n 2^-24 times the
sum of their magnitudes; here a thread adds at most 16 values (32 with both
vectors' halves) one after another and the rest is a tree of at most 10 levels
with at most 32 words at its end, so 80 steps bound every row sum.  With
T = mean |h|:
  mean   80 2^-24 T
  rstd   the mean's error shifts the deviations by d <= 80 2^-24 T, which adds d^2 to
         the variance (the deviations add up to 0); the rest is relative: half of 80 + 4 roundings
  y      half a step of bf16 (2^-8 of the value) and the errors of mean, rstd and three operations
"""
import numpy as np  # noqa: F401
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEPS = 80
EPS = 1e-5
BF, F32 = torch.bfloat16, torch.float32


def make(rows, cols, seed, std=1.0, offset=0.0, pad=0, shift=0):
    """A bf16 [rows, cols] tensor whose rows begin `shift` values behind an aligned place."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = torch.randn((rows, cols + pad + shift), generator=g, device="cuda") * std + offset
    return full.to(BF)[:, shift:shift + cols]


def params(cols, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ((torch.randn(cols, generator=g, device="cuda") * 0.3 + 1.0).to(dtype),
            (torch.randn(cols, generator=g, device="cuda") * 0.5).to(dtype))


def half_step(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


def forward64(h, w, b, eps=EPS):
    h = h.double()
    mean = h.mean(1, keepdim=True)
    rstd = 1.0 / ((h - mean).square().mean(1, keepdim=True) + eps).sqrt()
    xhat = (h - mean) * rstd
    return mean, rstd, xhat, xhat * w.double() + (0 if b is None else b.double())


def check_forward(h, w, b, y, stats, eps=EPS):
    mean, rstd, xhat, ref = forward64(h, w, b, eps)
    t = h.double().abs().mean(1, keepdim=True)
    d_mean = STEPS * U * t
    d_rstd = rstd * ((STEPS / 2 + 4) * U + (d_mean * rstd).square())
    if stats is not None:
        assert torch.all((stats[0][:, None].double() - mean).abs() <= d_mean)
        assert torch.all((stats[1][:, None].double() - rstd).abs() <= d_rstd)
    d_xhat = rstd * d_mean + xhat.abs() * (d_rstd / rstd + 3 * U)
    tol = 2.0 ** -8 * ref.abs() + 1.01 * w.double().abs() * d_xhat + 2 * U * ref.abs() + 2.0 ** -133
    assert torch.all((y.double() - ref).abs() <= tol), float(((y.double() - ref).abs() / tol).max())


SIZES = [(1, 1), (3, 7), (5, 64), (2, 255), (9, 256), (4, 257), (3, 513), (7, 1024), (5, 1531),
         (3, 2048), (2, 4095), (3, 4096), (2, 5000), (3, 8192), (2, 12289), (2, 16384), (700, 96),
         (1300, 1600), (2500, 136), (400, 1025)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, dtype):
    import quantised_gemm_gb300 as q
    x, (w, b) = make(rows, cols, 1), params(cols, dtype, 2)
    y, stats = torch.empty_like(x), torch.empty((2, rows), device="cuda")
    assert q.layer_norm(x, w, b, y, stats) is y
    check_forward(x, w, b, y, stats)
    y2 = torch.empty_like(x)
    q.layer_norm(x, w, None, y2)
    check_forward(x, w, None, y2, None)


@pytest.mark.parametrize("rows,cols,shift,pad", [(5, 64, 1, 0), (6, 1531, 0, 0), (6, 1531, 3, 2),
                                                 (4, 4096, 7, 1), (4, 4096, 8, 8), (3, 515, 2, 9),
                                                 (37, 250, 5, 0), (3, 9001, 4, 3), (2, 33, 6, 1)])
def test_forward_strided_unaligned_with_residual(rows, cols, shift, pad):
    import quantised_gemm_gb300 as q
    x, r = make(rows, cols, 3, pad=pad, shift=shift), make(rows, cols, 4, 3.0, pad=2 * pad, shift=pad)
    w, b = params(cols + 3, BF, 5)
    w, b = w[1:cols + 1], b[3:]
    full = torch.full((2, rows, cols + 16), 7.0, dtype=BF, device="cuda")
    y, h = full[0][:, 5:5 + cols], full[1][:, pad:pad + cols]
    want = full.clone()
    stats = torch.empty((2, rows), device="cuda")
    q.layer_norm(x, w, b, y, stats, residual=r, h=h)
    assert torch.equal(h, x + r)
    check_forward(h, w, b, y, stats)
    want[0][:, 5:5 + cols], want[1][:, pad:pad + cols] = y, h
    assert torch.equal(full, want)  # nothing beside the rows is written


@pytest.mark.parametrize("cols", [96, 1531, 4096])
def test_forward_in_place(cols):
    import quantised_gemm_gb300 as q
    x, r, (w, b) = make(70, cols, 6), make(70, cols, 7), params(cols, F32, 8)
    y, h = torch.empty_like(x), torch.empty_like(x)
    q.layer_norm(x, w, b, y, residual=r, h=h)
    for into in (0, 1):
        a = [x.clone(), r.clone()]
        y2 = torch.empty_like(x)
        q.layer_norm(a[0], w, b, y2, residual=a[1], h=a[into])
        assert torch.equal(a[into], h) and torch.equal(y2, y)
    a = x.clone()
    q.layer_norm(a, w, b, a)
    q.layer_norm(x, w, b, y)
    assert torch.equal(a, y)


def test_large_mean_and_constant_rows():
    import quantised_gemm_gb300 as q
    x, (w, b) = make(6, 4096, 9, std=1.0, offset=300.0), params(4096, F32, 10)
    x[2] = 5.0
    x[3] = 0.0
    x[4] = 3e38
    y, stats = torch.empty_like(x), torch.empty((2, 6), device="cuda")
    q.layer_norm(x, w, b, y, stats)
    ok = [0, 1, 2, 3, 5]
    check_forward(x[ok], w, b, y[ok], stats[:, ok])
    assert torch.equal(y[3], b.to(BF))


def test_nan_and_infinity_stay_in_their_rows():
    import quantised_gemm_gb300 as q
    x, (w, b) = make(9, 520, 11), params(520, BF, 12)
    clean = torch.empty_like(x)
    q.layer_norm(x, w, b, clean)
    x2 = x.clone()
    x2[1, 0], x2[4, 519], x2[7, 100] = float("nan"), float("inf"), float("-inf")
    y, amax = torch.empty_like(x), torch.empty(1, device="cuda")
    q.layer_norm(x2, w, b, y, None, q.Workspace(), y_amax=amax)
    bad = [1, 4, 7]
    assert torch.isnan(y[bad]).all() and torch.isnan(amax).all()
    ok = [0, 2, 3, 5, 6, 8]
    assert torch.equal(y[ok], clean[ok])


@pytest.mark.parametrize("rows,cols", [(0, 64), (1, 1), (33, 200), (9, 1531), (5000, 512), (4097, 2048)])
def test_amax_of_y_and_dx(rows, cols):
    import quantised_gemm_gb300 as q
    ws = q.Workspace()
    x, dy, (w, b) = make(rows, cols, 13), make(rows, cols, 14), params(cols, BF, 15)
    y, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty((2, rows), device="cuda")
    for _ in range(2):  # the words in the workspace are left as they were
        amax = torch.full((2,), -1.0, device="cuda")
        q.layer_norm(x, w, b, y, stats, ws, y_amax=amax[:1])
        q.layer_norm_backward(dy, x, w, stats, dx, None, None, ws, dx_amax=amax[1:])
        for got, t in zip(amax, (y, dx)):
            assert float(got) == (float(t.float().abs().max()) if rows else 0.0)


def check_backward(q, dy, x, w, stats, dx, dw, db, dres=None):
    mean, rstd = stats[0][:, None].double(), stats[1][:, None].double()
    xhat = (x.double() - mean) * rstd
    g = dy.double() * w.double()
    ref = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    # Row sums as above; g, xhat and the products are single roundings each.
    part = g.abs() + g.abs().mean(1, keepdim=True) + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True)
    tol = (STEPS + 10) * U * rstd * part
    if dres is not None:
        ref = ref + dres.double()
        tol = tol + U * dres.double().abs()
    tol = tol + 2.0 ** -8 * (ref.abs() + tol) + 2.0 ** -133
    assert torch.all((dx.double() - ref).abs() <= tol), float(((dx.double() - ref).abs() / tol).max())
    rows = x.shape[0]
    for got, terms in ((dw, dy.double() * xhat), (db, dy.double())):
        want = terms.sum(0)
        tol = (rows + 4) * U * terms.abs().sum(0) + 2.0 ** -133
        tol = tol + half_step(got.dtype) * (want.abs() + tol)
        assert torch.all((got.double() - want).abs() <= tol)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(rows, cols, dtype):
    import quantised_gemm_gb300 as q
    x, dy, (w, b) = make(rows, cols, 21), make(rows, cols, 22, 1e-2), params(cols, dtype, 23)
    y, stats, dx = torch.empty_like(x), torch.empty((2, rows), device="cuda"), torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    ws = q.Workspace()
    q.layer_norm(x, w, b, y, stats)
    q.layer_norm_backward(dy, x, w, stats, dx, dw, db, ws)
    check_backward(q, dy, x, w, stats, dx, dw, db)
    # The same bits again, and with a residual's gradient; only some of the outputs.
    dw2, db2, dx2, dres = torch.empty_like(w), torch.empty_like(w), torch.empty_like(x), make(rows, cols, 24)
    q.layer_norm_backward(dy, x, w, stats, None, dw2, db2, ws)
    assert torch.equal(dw, dw2) and torch.equal(db, db2)
    q.layer_norm_backward(dy, x, w, stats, dx2, None, db2, ws, dres=dres)
    check_backward(q, dy, x, w, stats, dx2, dw, db2, dres)
    q.layer_norm_backward(dy, x, w, stats, dx2, None, None, ws)
    assert torch.equal(dx2, dx)


@pytest.mark.parametrize("rows,cols,shift,pad", [(5, 64, 1, 0), (6, 1531, 3, 2), (4, 4096, 7, 1),
                                                 (700, 515, 2, 9), (3, 9001, 4, 3)])
def test_backward_strided_unaligned_in_place(rows, cols, shift, pad):
    import quantised_gemm_gb300 as q
    x, dy = make(rows, cols, 25, pad=pad, shift=shift), make(rows, cols, 26, pad=2, shift=pad)
    dres = make(rows, cols, 27, shift=1)
    w, b = params(cols, F32, 28)
    y, stats, ws = torch.empty_like(x), torch.empty((2, rows), device="cuda"), q.Workspace()
    q.layer_norm(x, w, b, y, stats)
    full = torch.full((rows, cols + 16), 7.0, dtype=BF, device="cuda")
    dx, want = full[:, 5:5 + cols], full.clone()
    dw, db = torch.empty_like(w), torch.empty_like(w)
    q.layer_norm_backward(dy, x, w, stats, dx, dw, db, ws, dres=dres)
    check_backward(q, dy, x, w, stats, dx, dw, db, dres)
    want[:, 5:5 + cols] = dx
    assert torch.equal(full, want)
    for t in (0, 1):
        into = [dy.clone(), dres.clone()]
        q.layer_norm_backward(into[0], x, w, stats, into[t], dw, db, ws, dres=into[1])
        assert torch.equal(into[t], dx)


def test_backward_against_differences():
    """<dx, u>, <dw, v> and <db, v> against central differences of sum(dy y) in 64 bits.  With eps of
    2^-12 the third derivative leaves a relative 2^-22 or so of terms of size 1; bf16 dx dominates."""
    import quantised_gemm_gb300 as q
    rows, cols = 40, 360
    x, dy, (w, b) = make(rows, cols, 31), make(rows, cols, 32), params(cols, F32, 33)
    y, stats, dx = torch.empty_like(x), torch.empty((2, rows), device="cuda"), torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    q.layer_norm(x, w, b, y, stats)
    q.layer_norm_backward(dy, x, w, stats, dx, dw, db, q.Workspace())
    g = torch.Generator(device="cuda").manual_seed(34)

    def loss(x, w, b):
        return float((dy.double() * forward64(x, w, b)[3]).sum())

    e = 2.0 ** -12
    u = torch.randn((rows, cols), generator=g, device="cuda").double()
    v = torch.randn(cols, generator=g, device="cuda").double()
    x64, w64, b64 = x.double(), w.double(), b.double()
    for got, grad, diff in ((dx, u, loss(x64 + e * u, w, b) - loss(x64 - e * u, w, b)),
                            (dw, v, loss(x, w64 + e * v, b) - loss(x, w64 - e * v, b)),
                            (db, v, loss(x, w, b64 + e * v) - loss(x, w, b64 - e * v))):
        terms = got.double() * grad
        # A value's half step, and 1e-3 of it for everything smaller.
        tol = (half_step(got.dtype) + 1e-5) * float(terms.abs().sum())
        assert abs(float(terms.sum()) - diff / (2 * e)) <= tol


def test_no_rows():
    import quantised_gemm_gb300 as q
    x, (w, b) = make(0, 40, 41), params(40, BF, 42)
    stats = torch.empty((2, 0), device="cuda")
    q.layer_norm(x, w, b, torch.empty_like(x), stats)
    dw, db = torch.ones_like(w), torch.ones_like(w)
    q.layer_norm_backward(x, x, w, stats, torch.empty_like(x), dw, db, q.Workspace())
    assert not dw.any() and not db.any()


def test_captured_and_replayed_on_another_stream():
    import quantised_gemm_gb300 as q
    rows, cols = 300, 1600
    x, dy, (w, b) = make(rows, cols, 51), make(rows, cols, 52), params(cols, BF, 53)
    norm = q.LayerNorm(rows, cols)
    res = make(rows, cols, 54)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        norm.forward(x, w, b, res)
        norm.backward(dy, res)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            norm.forward(x, w, b, res)
            norm.backward(dy, res)
    for seed in (55, 56):
        x.copy_(make(rows, cols, seed))
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm.h, x + res)
        check_forward(norm.h, w, b, norm.y, norm.stats)
        check_backward(q, dy, norm.h, w, norm.stats, norm.dx, norm.dw, norm.db, res)


@pytest.mark.parametrize("kind", ["fp8", "nvfp4"])
def test_between_linears(kind):
    """Linear, norm, Linear, linked and not: the same bits, as the maxima are the same."""
    import quantised_gemm_gb300 as q
    M, K, N = 272, 512, 768
    x, dy = make(M, K, 61), make(M, K, 62, 1e-3)
    w1, w2 = make(N, K, 63, 0.05), make(K, N, 64, 0.05)
    w, b = params(N, BF, 65)
    kept = []
    for linked in (False, True):
        if kind == "fp8":
            l1, l2 = q.Fp8Linear(M, K, N), q.Fp8Linear(M, N, K)
        else:
            l1, l2 = q.Fp4Linear(M, K, N), q.Fp4Linear(M, N, K)
        norm = q.LayerNorm(M, N)
        if linked:
            q.link_linears(norm, l2)
            q.link_linears(l1, norm)
            assert l2.sx.amax_algo == q.AMAX_PRECOMPUTED and l1.sdy.amax_algo == q.AMAX_PRECOMPUTED
        y = l2.forward(norm.forward(l1.forward(x, w1), w, b), w2)
        dx2, dw2 = l2.backward(dy)
        dx, dw, db = norm.backward(dx2)
        dx1, dw1 = l1.backward(dx)
        check_backward(q, dx2, l1.y, w, norm.stats, dx, dw, db)
        kept.append([t.clone() for t in (y, dx2, dw2, dx, dw, db, dx1, dw1, l2.sx.amax, l1.sdy.amax)])
    for a, c in zip(*kept):
        assert torch.equal(a, c)
    with pytest.raises(ValueError):
        q.link_linears(q.LayerNorm(M, N), q.LayerNorm(M, N))
    with pytest.raises(ValueError):
        q.link_linears(q.Fp4Linear(M, K, N), q.Fp8Linear(M, N, K))  # no amax from 4-bit products
    with pytest.raises(ValueError):
        q.link_linears(norm, q.Fp8Linear(M, N, K, scaling="delayed"))


def test_refusals():
    import quantised_gemm_gb300 as q
    x, (w, b) = make(4, 64, 71), params(64, BF, 72)
    y, stats, ws = torch.empty_like(x), torch.empty((2, 4), device="cuda"), q.Workspace()
    amax = torch.empty(1, device="cuda")
    q.layer_norm(x, w, b, y, stats)
    bad = [dict(y=torch.empty((4, 63), dtype=BF, device="cuda")), dict(w=w[:63]), dict(b=b.float()),
           dict(w=w.half()), dict(x=x.float()), dict(stats=stats[:1]), dict(residual=x), dict(h=y),
           dict(y_amax=amax), dict(y_amax=torch.empty(2, device="cuda"), ws=ws), dict(x=x.cpu()),
           dict(x=x.t()), dict(eps=-1.0), dict(eps=float("nan")), dict(b=b[::2])]
    for change in bad:
        args = dict(x=x, w=w, b=b, y=y, stats=stats, ws=None, eps=EPS, residual=None, h=None, y_amax=None)
        args.update(change)
        with pytest.raises((ValueError, TypeError, q.Fp8linError)):
            q.layer_norm(**args)
    wide = torch.empty((1, 16385), dtype=BF, device="cuda")
    with pytest.raises(q.Fp8linError):
        q.layer_norm(wide, wide[0], None, wide)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    for change in (dict(ws=None), dict(dw=dw.float()), dict(dx=dx[:3]), dict(dres=dx.float()),
                   dict(stats=stats.double()), dict(dx=None, dx_amax=amax), dict(db=dw[:5])):
        args = dict(dy=x, x=x, w=w, stats=stats, dx=dx, dw=dw, db=None, ws=ws, dres=None, dx_amax=None)
        args.update(change)
        with pytest.raises((ValueError, TypeError, q.Fp8linError)):
            q.layer_norm_backward(**args)
    norm = q.LayerNorm(4, 64)
    with pytest.raises(ValueError):
        norm.backward(x)
    with pytest.raises(TypeError):
        norm.forward(x, w.float(), None)
    norm.forward(x, w, b)
    with pytest.raises(ValueError):
        norm.forward(x[:3], w, b)
    with pytest.raises(ValueError):
        norm.backward(x)  # the forward before was refused


@pytest.mark.parametrize("cols", [96, 1531])
def test_forward_over_the_residual(cols):
    import quantised_gemm_gb300 as q
    x, r, (w, b) = make(70, cols, 81), make(70, cols, 82), params(cols, F32, 83)
    y, h = torch.empty_like(x), torch.empty_like(x)
    q.layer_norm(x, w, b, y, residual=r, h=h)
    h2 = torch.empty_like(h)
    q.layer_norm(x, w, b, r, residual=r, h=h2)
    assert torch.equal(r, y) and torch.equal(h2, h)


def test_a_norm_delivers_its_maximum_to_one_layer():
    """A second layer would leave the first one's scale to a maximum that nothing writes."""
    import quantised_gemm_gb300 as q
    norm, first, second = q.LayerNorm(32, 64), q.Fp8Linear(32, 64, 96), q.Fp8Linear(32, 64, 96)
    q.link_linears(norm, first)
    q.link_linears(norm, first)
    with pytest.raises(ValueError):
        q.link_linears(norm, second)
    assert second.sx.amax_algo != q.AMAX_PRECOMPUTED
    before, other = q.Fp8Linear(32, 128, 64), q.Fp8Linear(32, 128, 64)
    q.link_linears(before, norm)
    with pytest.raises(ValueError):
        q.link_linears(other, norm)
    assert other.sdy.amax_algo != q.AMAX_PRECOMPUTED and other.y_amax_to is None
