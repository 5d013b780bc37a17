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


@pytest.mark.parametrize("rows", [20, 100, 700, 5000])
@pytest.mark.parametrize("k,n,rank", [(200, 104, 16), (99, 57, 6), (256, 320, 64), (72, 136, 128), (40, 64, 32)])
def test_sums_that_cancel_are_exact(k, n, rank, rows):
    """Whole numbers of 16 bits as h and dh, which hi + lo holds.  From column 3 on they meet 1 and -1 in
    pairs (of ranks in y and dx, of rows in dA and dB) that cancel but for some units; every product and
    partial sum is a whole number below 2^24, and in columns 0 to 2 of y and dx at most 2^23 times 1 or 256,
    so the results are the formulas' rounded once.  A bit of lo lost would be seen."""
    import quantised_gemm_gb300 as q
    g = torch.Generator(device="cuda").manual_seed(91)
    ints = lambda lo, hi, shape: torch.randint(lo, hi + 1, shape, generator=g, device="cuda").float()  # noqa: E731
    zeros = lambda *shape: torch.zeros(shape, dtype=BF, device="cuda")  # noqa: E731
    a, b, x, dy = zeros(2, rank, k), zeros(2, n, rank), zeros(rows, k), zeros(rows, n)
    # h_j = 256 x0 + x1, and x2 more for odd j; B has ones of changing sign, and so has A from column 3 on.
    a[:, :, 0], a[:, :, 1], a[:, 1::2, 2] = 256.0, 1.0, 1.0
    sign = torch.ones(rank, device="cuda")
    sign[1::2] = -1.0
    b[:, 3:, :] = sign
    a[:, :, 3:] = sign[:, None]
    b[:, 0], b[:, 1], b[:, 2, 1::2] = 256.0, 1.0, 1.0
    pair = torch.arange(rows, device="cuda") // 2
    index = torch.randint(0, 2, (rows // 2 + 1,), generator=g, device="cuda")[pair].to(torch.int32)
    one = torch.where(torch.arange(rows, device="cuda") % 2 == 0, 1.0, -1.0)  # the rows of a pair
    for t in (x, dy):
        t[:, 0], t[:, 1] = ints(128, 250, (rows // 2 + 1,))[pair], ints(0, 250, (rows // 2 + 1,))[pair]
        t[:, 2] = ints(1, 3, (rows,))
    x[:, 3:], dy[:, 3:] = one[:, None], one[:, None]
    bank = q.Adapters(a, b, torch.ones(2, device="cuda"))
    c = Case(rows, k, n, rank, 2)  # its buffers
    c.x, c.dy, c.bank, c.index = x, dy, bank, index
    y = torch.empty((rows, n), dtype=BF, device="cuda")
    c.forward(y, base=None)
    h = torch.zeros((rows, rank), dtype=torch.float64, device="cuda")
    dh = torch.zeros_like(h)
    ref, dref = (torch.zeros((rows, cols), dtype=torch.float64, device="cuda") for cols in (n, k))
    dx, da, db = c.like()
    c.backward(dx, da, db, base=None)
    for i, r in enumerate(c.groups()):
        h[r], dh[r] = x[r].double() @ a[i].double().t(), dy[r].double() @ b[i].double()
        ref[r], dref[r] = h[r] @ b[i].double().t(), dh[r] @ a[i].double()
        assert torch.equal(da[i][:, 3:], (dh[r].t() @ x[r].double())[:, 3:].to(BF)), "dA"
        assert torch.equal(db[i][3:], (dy[r].double().t() @ h[r])[3:].to(BF)), "dB"
    assert float(h.abs().max()) < 2 ** 16 and float(dh.abs().max()) < 2 ** 16
    assert torch.equal(c.h.double(), h) and torch.equal(c.dh.double(), dh)
    assert torch.equal(y, ref.to(BF)) and torch.equal(dx, dref.to(BF))
