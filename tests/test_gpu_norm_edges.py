"""The layer norm where rows are constant or leave fp32's range."""
import pytest
import torch

from test_gpu_norm import BF, F32, make, params

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
