"""The layer norm, the 4-bit Linear and the adapters beside it as a program uses them
together: a batch served from a kept 4-bit weight, and a training step of the
adapters with that weight frozen."""
import pytest
import torch

from test_gpu_adapters import Case
from test_gpu_norm import check_backward, check_forward, make, params

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("rows", [1, 24, 200])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_serving(rows, fmt):
    """Residual and norm, then the Linear of a kept weight with an adapter a request."""
    import quantised_gemm_gb300 as q
    k, n = 416, 608
    fmt = q.NVFP4 if fmt == "nv" else q.MXFP4
    c = Case(rows, k, n, 16, 5, "random", 3)
    hidden, block, (w, b) = make(rows, k, 4), make(rows, k, 5), params(k, BF, 6)
    ws = q.Workspace()
    w4, x4 = q.Fp4Tensor(n, k, fmt), q.Fp4Tensor(rows, k, fmt)
    q.fp4_quantise(make(n, k, 7, 0.05), w4, None, ws)
    normed = torch.empty_like(hidden)
    y, plain = (torch.empty((rows, n), dtype=BF, device="cuda") for _ in range(2))

    def token():
        q.layer_norm(block, w, b, normed, None, ws, residual=hidden, h=hidden)
        q.fp4_linear(normed, x4, w4, y, ws, adapters=c.bank, index=c.index, h=c.h)

    before = hidden.clone()
    token()
    assert torch.equal(hidden, before + block)
    check_forward(hidden, w, b, normed, None)
    q.fp4_linear(normed, x4, w4, plain, ws)
    c.x = normed
    c.check_forward(y, base=plain)
    # The same through a graph, on the sorted rows where there are many.
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        token()
    hidden.copy_(before)
    want = y.clone()
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    for bad in (dict(adapters=c.bank), dict(index=c.index), dict(h=c.h), dict(adapters=c.bank, index=c.index),
                dict(adapters=c.bank, index=c.index[:0], h=c.h)):
        with pytest.raises((ValueError, q.Fp8linError)):
            q.fp4_linear(normed, x4, w4, y, ws, **bad)


@pytest.mark.parametrize("kind", ["fp8", "fp4"])
def test_training_step(kind):
    """norm -> frozen Linear + adapters; backward through all, dx of the Linear as the base; the
    adapters' gradients clipped together with the norm's."""
    import quantised_gemm_gb300 as q
    rows, k, n = 272, 256, 384
    c = Case(rows, k, n, 8, 3, "runs", 13)
    x, (w, b), weight, dy = make(rows, k, 14), params(k, torch.float32, 15), make(n, k, 16, 0.05), make(rows, n, 17, 1e-2)
    norm = q.LayerNorm(rows, k, param_dtype=torch.float32)
    lin = q.Fp8Linear(rows, k, n) if kind == "fp8" else q.Fp4Linear(rows, k, n)
    q.link_linears(norm, lin)
    ws, route = q.Workspace(), q.AdapterRoute(rows, 3).set(c.index)
    c.x = norm.forward(x, w, b)
    check_forward(x, w, b, c.x, norm.stats)
    base = lin.forward(c.x, weight).clone()
    y = q.adapter_linear(c.x, c.index, c.bank, lin.y, c.h, ws, base=lin.y, route=route)
    c.check_forward(y, base=base)
    dx, _ = lin.backward(dy, need_dw=False)
    dbase, c.dy = dx.clone(), dy
    _, da, db = c.like()
    q.adapter_backward(dy, c.x, c.h, c.index, c.bank, c.dh, dx, da, db, ws, base=dx, route=route)
    c.check_backward(dx, da, db, base=dbase)
    dxn, dw, dbias = norm.backward(dx)
    check_backward(q, dx, x, w, norm.stats, dxn, dw, dbias)
    grads = [da, db, dw, dbias]
    total = sum(float(g.double().square().sum()) for g in grads) ** 0.5
    out = torch.empty(1, device="cuda")
    q.clip_grad_norm(grads, total / 2, out, ws)
    assert abs(float(out) - total) <= 1e-5 * total


def test_a_route_without_adapters_is_refused():
    import quantised_gemm_gb300 as q
    x, ws, y = make(8, 64, 21), q.Workspace(), torch.empty((8, 32), dtype=BF, device="cuda")
    w4, x4 = q.Fp4Tensor(32, 64, q.NVFP4), q.Fp4Tensor(8, 64, q.NVFP4)
    with pytest.raises(ValueError):
        q.fp4_linear(x, x4, w4, y, ws, route=q.AdapterRoute(8, 2))
