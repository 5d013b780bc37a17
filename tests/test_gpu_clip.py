"""The global gradient norm and the clipping on the GPU against fp64."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def grads_of(sizes, dtypes, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * scale).to(dtypes[i % len(dtypes)])
            for i, s in enumerate(sizes)]


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check(q, grads, max_norm, outs=None):
    """One call against fp64.  A thread adds at most 32 squares at a time in
    fp32, each sum within 128 * 2^-24 of its squares' total, so the
    norm within half that; the factor adds three roundings, the value one."""
    want = norm64(grads)
    before = [g.clone() for g in grads]
    norm = torch.full((1,), -1.0, device="cuda")
    q.clip_grad_norm(grads, max_norm, norm, q.Workspace(), outs=outs)
    tol = 64 * 2.0 ** -24 + 2.0 ** -23
    assert abs(float(norm) - want) <= tol * want
    coef = min(1.0, max_norm / (want + 1e-6))
    for b, o in zip(before, outs if outs is not None else grads):
        ref = b.double() * coef
        ulp = 2.0 ** -8 if o.dtype == torch.bfloat16 else 2.0 ** -24
        assert torch.all((o.double() - ref).abs() <= (ulp + tol + 4 * 2.0 ** -24) * ref.abs()
                         + 2.0 ** -133)
    return norm


SIZES = [[(1,)], [(7,), (1,), (33, 3)], [(16384,)], [(16385,), (5,)], [(1600, 129), (1600,), (64, 64)],
         [(3_000_001,)], [(100 + i,) for i in range(40)], [(3,)] * 1000 + [(70000,)] * 3]


@pytest.mark.parametrize("dtypes", [(torch.bfloat16,), (torch.float32,),
                                    (torch.bfloat16, torch.float32)], ids=["bf16", "f32", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
def test_clip_in_place(sizes, dtypes):
    import quantised_gemm_gb300 as q
    check(q, grads_of(sizes, dtypes, 3), 0.5)


@pytest.mark.parametrize("to", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("frm", [torch.bfloat16, torch.float32])
def test_clip_into_other_tensors(frm, to):
    import quantised_gemm_gb300 as q
    sizes = [(257, 31), (9,), (40000,)]
    grads = grads_of(sizes, (frm,), 4)
    kept = [g.clone() for g in grads]
    outs = [torch.full(s, 9.0, dtype=to, device="cuda") for s in sizes]
    check(q, grads, 1.0, outs)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))


def test_below_the_largest_norm_nothing_changes():
    import quantised_gemm_gb300 as q
    grads = grads_of([(1000,), (77, 3)], (torch.bfloat16, torch.float32), 5)
    kept = [g.clone() for g in grads]
    check(q, grads, 1e6)
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))


def test_unaligned_and_transposed_gradients():
    import quantised_gemm_gb300 as q
    base = torch.randn(50_001, device="cuda")
    half = base.to(torch.bfloat16)
    m = torch.randn(65, 33, device="cuda").to(torch.bfloat16)
    grads = [base[1:], half[3:20_000], half[20_001:], m.t()]
    check(q, grads, 0.25)
    outs = [torch.empty_like(g, dtype=torch.float32) for g in grads]
    assert outs[3].stride() == m.t().stride()
    check(q, grads, 0.125, outs)


def test_norm_is_the_same_bits_every_time():
    import quantised_gemm_gb300 as q
    grads = grads_of([(1_234_567,), (89,), (300, 1000)], (torch.float32,), 6)
    ws, norm = q.Workspace(), torch.empty(1, device="cuda")
    got = {int(q.grad_norm(grads, norm, ws).view(torch.int32)) for _ in range(5)}
    assert len(got) == 1


def test_parts_equal_the_whole():
    import quantised_gemm_gb300 as q
    a = grads_of([(5000,), (31,)], (torch.bfloat16,), 7)
    b = [g.clone() for g in a]
    n1, n2, ws = torch.empty(1, device="cuda"), torch.empty(1, device="cuda"), q.Workspace()
    q.clip_grad_norm(a, 0.1, n1, ws)
    q.grad_norm(b, n2, ws)
    q.clip_grads(b, 0.1, n2)
    assert torch.equal(n1, n2) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_large_values_do_not_overflow():
    import quantised_gemm_gb300 as q
    g = [torch.full((5000,), 1e20, device="cuda"), torch.full((33,), -3e19, dtype=torch.bfloat16,
                                                               device="cuda")]
    norm = q.grad_norm(g, torch.empty(1, device="cuda"), q.Workspace())
    assert abs(float(norm) / norm64(g) - 1) < 1e-6


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1e-13, 1e-20, 1e-30, 1e-37])
def test_small_values_do_not_underflow(scale, dtype):
    import quantised_gemm_gb300 as q
    grads = grads_of([(5000,), (333, 7), (3,)], (dtype,), 8, scale)
    grads.append(torch.zeros(100_000, dtype=dtype, device="cuda"))
    want = norm64(grads)
    norm = torch.empty(1, device="cuda")
    q.grad_norm(grads, norm, q.Workspace())
    assert abs(float(norm) - want) <= (64 * 2.0 ** -24 + 2.0 ** -23) * want


def test_small_values_beside_large_ones():
    import quantised_gemm_gb300 as q
    grads = grads_of([(5000,)], (torch.float32,), 9, 1e-25) + \
        grads_of([(3000,)], (torch.float32,), 10, 1e18) + grads_of([(4000,)], (torch.float32,), 11)
    for part in (grads, grads[::2], grads[:1], grads[1:]):
        norm = torch.empty(1, device="cuda")
        q.grad_norm(part, norm, q.Workspace())
        want = norm64(part)
        assert abs(float(norm) - want) <= (64 * 2.0 ** -24 + 2.0 ** -23) * want


def test_empty_lists_and_tensors():
    import quantised_gemm_gb300 as q
    ws = q.Workspace()
    for grads in ([], [torch.empty(0, device="cuda")],
                  [torch.empty(0, device="cuda", dtype=torch.bfloat16), torch.empty((0, 5), device="cuda")]):
        norm = torch.full((1,), 3.0, device="cuda")
        q.clip_grad_norm(grads, 1.0, norm, ws)
        assert float(norm) == 0
    g = [torch.empty(0, device="cuda"), torch.tensor([3.0, 4.0], device="cuda"), torch.empty(0, device="cuda")]
    norm = torch.empty(1, device="cuda")
    q.clip_grad_norm(g, 1.0, norm, ws)
    assert float(norm) == 5 and abs(float(g[1][0]) - 0.6) < 1e-6


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_and_infinity(dtype):
    import quantised_gemm_gb300 as q
    ws = q.Workspace()
    for bad, want in ((float("nan"), torch.isnan), (float("inf"), torch.isinf)):
        g = [torch.ones(1000, dtype=dtype, device="cuda"), torch.ones(10, dtype=dtype, device="cuda")]
        g[0][500] = bad
        norm = torch.empty(1, device="cuda")
        q.clip_grad_norm(g, 1.0, norm, ws)
        assert want(norm).all()
        if math.isnan(bad):
            assert torch.isnan(g[0]).all() and torch.isnan(g[1]).all()
        else:  # a factor of zero
            assert (g[1] == 0).all() and torch.isnan(g[0][500]) and (g[0][:500] == 0).all()


def test_zero_gradients():
    import quantised_gemm_gb300 as q
    g = [torch.zeros(100, device="cuda")]
    norm = q.clip_grad_norm(g, 1.0, torch.empty(1, device="cuda"), q.Workspace())
    assert float(norm) == 0 and (g[0] == 0).all()


def test_a_call_on_another_stream():
    import quantised_gemm_gb300 as q
    side, ws = torch.cuda.Stream(), q.Workspace()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = [torch.randn(100_000, device="cuda")]
        want = norm64(g)
        norm = torch.empty(1, device="cuda")
        q.clip_grad_norm(g, 1.0, norm, ws)
    side.synchronize()
    assert abs(float(norm) / want - 1) < 1e-5 and abs(norm64(g) - 1) < 1e-5


def test_python_refusals():
    import quantised_gemm_gb300 as q
    norm, ws = torch.empty(1, device="cuda"), q.Workspace()
    x = torch.ones(8, device="cuda")
    with pytest.raises(TypeError):
        q.grad_norm([x.double()], norm, ws)
    with pytest.raises(ValueError):
        q.grad_norm([x.cpu()], norm, ws)
    with pytest.raises(ValueError):
        q.grad_norm([x[::2]], norm, ws)
    with pytest.raises(ValueError):
        q.grad_norm([x], torch.empty(2, device="cuda"), ws)
    with pytest.raises(ValueError):
        q.clip_grad_norm([x], 1.0, norm, ws, outs=[])
    with pytest.raises(ValueError):
        q.clip_grad_norm([x], 1.0, norm, ws, outs=[torch.empty(9, device="cuda")])
    with pytest.raises(ValueError):
        q.clip_grad_norm([x.view(2, 4)], 1.0, norm, ws, outs=[torch.empty(4, 2, device="cuda").t()])
    with pytest.raises(q.Fp8linError):
        q.clip_grad_norm([x], -1.0, norm, ws)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("in_place", [True, False])
def test_an_infinite_largest_norm_clips_nothing(dtype, in_place):
    import quantised_gemm_gb300 as q
    ws = q.Workspace()
    for special in (1.0, float("inf"), float("-inf"), float("nan")):
        g = [torch.randn(3000, device="cuda").to(dtype), torch.ones(10, dtype=dtype, device="cuda")]
        g[0][77] = special
        kept = [t.clone() for t in g]
        outs = None if in_place else [torch.empty_like(t) for t in g]
        norm = torch.empty(1, device="cuda")
        q.clip_grad_norm(g, float("inf"), norm, ws, outs=outs)
        assert math.isnan(float(norm)) if math.isnan(special) else math.isinf(float(norm)) == math.isinf(special)
        for got, was in zip(g if in_place else outs, kept):
            if math.isnan(special):
                assert torch.isnan(got).all()
            else:
                assert torch.equal(got, was)
        q.clip_grads(kept, float("inf"), norm)
        if not math.isnan(special):
            assert float(kept[0][77]) == special


def test_zero_gradients_stay_zero_without_room():
    import quantised_gemm_gb300 as q
    g, norm = [torch.zeros(100, device="cuda")], torch.empty(1, device="cuda")
    for outs in (None, [torch.ones(100, device="cuda")]):
        q.clip_grad_norm(g, 0.0, norm, q.Workspace(), outs=outs, eps=0.0)
        assert float(norm) == 0 and ((g if outs is None else outs)[0] == 0).all()
