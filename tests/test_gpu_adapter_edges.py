"""The adapters where buffers are shared, numbers are infinite and sums cancel."""
import pytest
import torch

from test_gpu_adapters import Case

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("rows,k,n,rank,count", [(256, 512, 512, 16, 1), (700, 264, 321, 12, 4), (1500, 520, 1024, 64, 3)])
def test_batches_in_turn_through_the_same_buffers(rows, k, n, rank, count):
    """Two batches' passes one after another, with one dh, workspace and set of outputs: each call finds
    what the call before it left in them."""
    cases = [Case(rows, k, n, rank, count, kind, seed) for kind, seed in (("random", 41), ("runs", 51))]
    y, out = torch.empty((rows, n), dtype=BF, device="cuda"), cases[0].like()
    want = []
    for c in cases:
        c.forward(y)
        c.backward(*out)
        torch.cuda.synchronize()
        c.check_backward(*out)
        want.append([t.clone() for t in out])
    cases[1].ws, cases[1].dh = cases[0].ws, cases[0].dh
    got = []
    for _ in range(6):
        for c in cases:
            c.backward(*out)
            got.append([t.clone() for t in out])
    torch.cuda.synchronize()
    for i, one in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(one, want[i % 2]))


def infinite_row(rank, rows=40, k=200, n=104):
    """Rows of which number 3 has an infinity that meets A of one sign and B of one sign: h and y of it
    are infinities of known signs."""
    c = Case(rows, k, n, rank, 2, "random", 61)
    c.index[:4] = 1
    c.x[3, 77] = float("inf")
    a, b = c.bank.a, c.bank.b
    a[1, :, 77] = a[1, :, 77].abs() + 0.01
    a[1, ::2, 77] *= -1.0
    b[1] = b[1].abs() + 0.01
    b[1, :, ::2] *= -1.0  # s h B is +inf for every rank
    return c


@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("rank", [3, 8, 12, 20, 24, 33, 40, 100])
def test_an_infinity_in_x_is_one_in_y(rank, rows):
    """In one launch (rank 100: 16 rows) and on the sorted rows alike, also where the ranks end inside a tile."""
    c = infinite_row(rank, 16 if rank == 100 and rows == 40 else rows)
    y = torch.empty((c.rows, c.n), dtype=BF, device="cuda")
    c.forward(y)
    sign = torch.ones(rank, device="cuda")
    sign[::2] = -1.0
    assert torch.equal(c.h[3], sign * float("inf"))
    assert torch.equal(y[3].float(), torch.full((c.n,), float("inf"), device="cuda"))
    assert torch.isfinite(y[:3]).all() and torch.isfinite(y[4:]).all()
