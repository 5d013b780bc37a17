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


def signed_infinity(v):
    return torch.where(v == 0, torch.nan, torch.sign(v) * float("inf"))


@pytest.mark.parametrize("rows", [16, 40, 300, 3000])
@pytest.mark.parametrize("k,n,rank", [(200, 104, 16), (200, 101, 16), (192, 200, 8), (256, 512, 64), (130, 77, 33), (64, 72, 128), (321, 97, 5)])
def test_an_infinity_in_a_bank(k, n, rank, rows):
    """An infinity of B or A is one of the sign of what it is multiplied with, whatever bits that has:
    in its column, and the other columns keep theirs."""
    c = Case(rows, k, n, rank, 2, "random", 71)
    y, y2 = (torch.empty((rows, n), dtype=BF, device="cuda") for _ in range(2))
    c.x[1::3, 1:] = 0.0  # of these rows h has only bf16's bits
    c.forward(y)
    dx, da, db = c.like()
    c.backward(dx, da, db)
    has = c.index == 1
    ranks = (rank - 1, rank // 2)
    cols = (n - 1, n // 3)
    for j, col, sign in zip(ranks, cols, (1.0, -1.0)):
        c.bank.b[1, col, j] = sign * float("inf")
    c.forward(y2)
    want = y.float()
    for j, col, sign in zip(ranks, cols, (1.0, -1.0)):
        want[has, col] = signed_infinity(sign * c.h[has, j])
    assert torch.equal(y2.float().nan_to_num(5.0, 7.0, -7.0), want.nan_to_num(5.0, 7.0, -7.0))
    c.bank.b[1, cols[0], ranks[0]] = c.bank.b[1, cols[1], ranks[1]] = 0.0
    dx2 = c.like()[0]
    c.backward(dx, None, None)
    cols = (k - 1, k // 3)
    for j, col, sign in zip(ranks, cols, (1.0, -1.0)):
        c.bank.a[1, j, col] = sign * float("inf")
    c.backward(dx2, None, None)
    want = dx.float()
    for j, col, sign in zip(ranks, cols, (1.0, -1.0)):
        want[has, col] = signed_infinity(sign * c.dh[has, j])
    assert torch.equal(dx2.float().nan_to_num(5.0, 7.0, -7.0), want.nan_to_num(5.0, 7.0, -7.0))


@pytest.mark.parametrize("rows", [16, 100, 700, 3000])
@pytest.mark.parametrize("k,n,rank", [(200, 104, 16), (201, 101, 16), (192, 200, 8), (256, 512, 64), (130, 77, 33), (64, 72, 128), (321, 97, 5)])
def test_an_infinity_in_x_or_dy_is_seen_in_the_gradients(k, n, rank, rows):
    """An infinity in x makes its column of dA infinite or NaN, one in dy its row of dB, in the adapter of
    that row of the batch; the other numbers keep their bits."""
    c = Case(rows, k, n, rank, 3, "random", 81)
    c.index[7], c.index[11] = 1, 2
    c.x[1::3, 1:] = 0.0
    c.forward(torch.empty((rows, n), dtype=BF, device="cuda"))
    _, da, db = c.like()
    c.backward(None, da, db)
    _, da2, db2 = c.like()
    c.x[7, k // 3], c.x[11, k - 1] = float("inf"), float("-inf")
    c.backward(None, da2, db2)
    seen = torch.zeros(da.shape, dtype=torch.bool, device="cuda")
    seen[1, :, k // 3] = seen[2, :, k - 1] = True
    assert torch.equal(db2, db)
    assert torch.equal(~torch.isfinite(da2), seen) and torch.equal(da2[~seen], da[~seen])
    c.x[7, k // 3] = c.x[11, k - 1] = 0.0
    c.dy[7, n // 3], c.dy[11, n - 1] = float("-inf"), float("inf")
    c.backward(None, da2, db2)
    seen = torch.zeros(db.shape, dtype=torch.bool, device="cuda")
    seen[1, n // 3] = seen[2, n - 1] = True
    assert torch.equal(~torch.isfinite(db2), seen) and torch.equal(db2[~seen], db[~seen])
    assert torch.equal(da2[0], da[0]) and not torch.isfinite(da2[1:]).any()
