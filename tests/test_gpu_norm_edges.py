"""The layer norm where rows are constant or leave fp32's range."""
import pytest
import torch

from test_gpu_norm import BF, F32, check_backward, check_forward, make, params

pytestmark = pytest.mark.gpu

COLS = [1, 3, 7, 100, 257, 777, 1531, 1600, 2047, 4099, 5000, 9001, 16383, 16384]


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("cols", COLS)
def test_rows_of_equal_values(cols, shift):
    """Equal bf16 values have 8 bits and their number at most 14, so every partial sum is exact in fp32,
    the mean is the value, the deviations are 0 and y is b."""
    import quantised_gemm_gb300 as q
    values = torch.tensor([1000.0, -77.5, 3.140625, 0.1, 65280.0, 1e30, -1e-30], device="cuda").to(BF)
    x = make(len(values), cols, 1, shift=shift)
    x.copy_(values[:, None].expand(-1, cols))
    w, b = params(cols, F32, 2)
    y, stats = torch.empty_like(x), torch.empty((2, len(values)), device="cuda")
    q.layer_norm(x, w, b, y, stats)
    assert torch.equal(stats[0], values.float())
    assert torch.all((stats[1].double() * 1e-5 ** 0.5 - 1.0).abs() <= 2.0 ** -22)  # eps and the root
    assert torch.equal(y, b.to(BF).expand_as(y))


def wide_rows(cols, shift=0):
    """Finite rows whose sums or squares leave fp32's range, each between rows that do not."""
    x = make(20, cols, 3, shift=shift)
    f = x.float()
    f[1] *= 1e20
    f[3] *= 3e30
    f[5] = (f[5] * 1e38).clamp(-3e38, 3e38)
    f[7] = 3e38
    f[9] = 3e38
    f[9, ::2] = -3e38
    f[11, cols // 2] = -3.3e38
    f[13] = 1e38 + f[13] * 1e36
    f[15] = f[15] * 1e-3 + 3e37
    f[17] = 2.5e38
    f[17, 0] = 2.4e38
    x.copy_(f.to(BF))
    return x


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("cols,shift", [(96, 0), (96, 1), (300, 0), (520, 0), (1531, 0), (1600, 0), (4096, 0), (4096, 3), (5001, 0),
                                        (8192, 0), (9001, 2), (16384, 0)])
def test_rows_beyond_the_range_of_their_squares(cols, shift, residual):
    """Statistics and y of finite rows are those of the formula; the other rows keep their bits."""
    import quantised_gemm_gb300 as q
    x, (w, b) = wide_rows(cols, shift), params(cols, F32, 4)
    y, stats = torch.empty_like(x), torch.empty((2, 20), device="cuda")
    if residual:
        r, h = make(20, cols, 5, 1e-3), make(20, cols, 6, shift=1)
        q.layer_norm(x, w, b, y, stats, residual=r, h=h)
        assert torch.equal(h, x + r)
    else:
        r, h = None, x
        q.layer_norm(x, w, b, y, stats)
    equal = 7  # and the others have deviations
    ok = [i for i in range(20) if i != equal]
    check_forward(h[ok], w, b, y[ok], stats[:, ok])
    assert torch.equal(y[equal], b.to(BF)) and stats[0, equal] == h[equal, 0].float()
    assert abs(float(stats[1, equal]) * 1e-5 ** 0.5 - 1.0) <= 2.0 ** -22
    calm = [i for i in range(20) if i % 2 == 0 or i == 19]
    x2 = x.clone()
    x2[[i for i in range(20) if i not in calm]] = 1.0
    y2, stats2 = torch.empty_like(y), torch.empty_like(stats)
    q.layer_norm(x2, w, b, y2, stats2, residual=r, h=None if r is None else torch.empty_like(x2))
    assert torch.equal(y2[calm], y[calm]) and torch.equal(stats2[:, calm], stats[:, calm])
    into = x.clone()  # in place
    q.layer_norm(into, w, b, into, residual=r, h=None if r is None else into)
    assert torch.equal(into, y)


@pytest.mark.parametrize("cols,shift", [(96, 0), (1531, 0), (4096, 3), (9001, 2), (16384, 0)])
def test_the_backward_of_such_rows(cols, shift):
    import quantised_gemm_gb300 as q
    x, dy, (w, b) = wide_rows(cols, shift), make(20, cols, 7, 1e-2), params(cols, F32, 8)
    y, stats, dx = torch.empty_like(x), torch.empty((2, 20), device="cuda"), torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    q.layer_norm(x, w, b, y, stats)
    q.layer_norm_backward(dy, x, w, stats, dx, dw, db, q.Workspace())
    check_backward(q, dy, x, w, stats, dx, dw, db)
