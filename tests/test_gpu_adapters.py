"""Low-rank adapters on the GPU against the formulas in 64 bits.

Bounds.  A product of two bf16 numbers is exact in fp32.  A tensor-core step adds
16 products to a sum; with every addend cut to the largest one's last bit that is
off by at most 17 2^-23 < 2^-18 of the magnitudes' sum S, and a warp does at most
K / 128 such steps one after another (8 warps, 32 columns and two steps a turn),
and a few more additions follow: h is off by at most (K / 128 + 8) 2^-18 S.  A number
that goes in as hi + lo is off by 2^-17 of it.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
STEP = 2.0 ** -18


def normal(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def padded(shape, seed, std, shift, pad):
    return normal((shape[0], shape[1] + shift + pad), seed, std)[:, shift:shift + shape[1]]


def make_index(rows, count, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "random":
        index = torch.randint(-1, count, (rows,), generator=g, device="cuda")
    elif kind == "runs":
        index = torch.randint(-1, count, (rows // 40 + 1,), generator=g, device="cuda").repeat_interleave(40)[:rows]
    elif kind == "none":
        index = torch.full((rows,), -1, device="cuda")
    elif kind == "same":
        index = torch.full((rows,), count - 1, device="cuda")
    else:  # numbers that name no adapter
        bad = torch.tensor([-5, count, 1 << 30, -(1 << 31), 0], device="cuda")
        index = bad[torch.randint(0, 5, (rows,), generator=g, device="cuda")]
    return index.to(torch.int32)


class Case:
    def __init__(self, rows, k, n, rank, count, kind="random", seed=1, shift=0, pad=0):
        import quantised_gemm_gb300 as q
        self.q, self.rows, self.k, self.n, self.rank, self.count = q, rows, k, n, rank, count
        self.x = padded((rows, k), seed, 1.0, shift, pad)
        self.base = padded((rows, n), seed + 1, 1.0, pad, shift)
        self.dy = padded((rows, n), seed + 2, 1e-2, shift, 1)
        self.dbase = padded((rows, k), seed + 3, 1e-2, pad, 2)
        self.bank = q.Adapters(normal((count, rank, k), seed + 4, k ** -0.5), normal((count, n, rank), seed + 5, 0.1),
                               torch.rand(count, device="cuda") + 0.5)
        self.index = make_index(rows, count, kind, seed + 6)
        self.h = torch.full((rows, rank), 9.0, device="cuda")
        self.dh = torch.full((rows, rank), 9.0, device="cuda")
        self.ws = q.Workspace()

    def forward(self, y, base="own", route=None):
        return self.q.adapter_linear(self.x, self.index, self.bank, y, self.h, self.ws,
                                     base=self.base if base == "own" else base, route=route)

    def backward(self, dx, da, db, base="own", h=None, route=None):
        return self.q.adapter_backward(self.dy, self.x, self.h if h is None else h, self.index, self.bank, self.dh, dx,
                                       da, db, self.ws, base=self.dbase if base == "own" else base, route=route)

    def groups(self):
        return [(self.index == i).nonzero()[:, 0] for i in range(self.count)]

    def check_forward(self, y, base="own"):
        base = self.base if base == "own" else base
        ref = torch.zeros((self.rows, self.n), dtype=torch.float64, device="cuda") if base is None else base.double()
        off = torch.zeros_like(ref)
        href, hoff = torch.zeros_like(self.h, dtype=torch.float64), torch.zeros_like(self.h, dtype=torch.float64)
        none = torch.ones(self.rows, dtype=torch.bool, device="cuda")
        for i, r in enumerate(self.groups()):
            x, a, b, s = self.x[r].double(), self.bank.a[i].double(), self.bank.b[i].double(), float(self.bank.scale[i])
            href[r], hoff[r] = x @ a.t(), (self.k / 128 + 8) * STEP * (x.abs() @ a.abs().t())
            ref[r] += s * (href[r] @ b.t())
            # hi + lo, the steps over the ranks and the product with s.
            off[r] = s * ((hoff[r] + (2.0 ** -17 + 2.0 ** -23 + (self.rank / 8 + 2) * STEP) * href[r].abs()) @ b.abs().t())
            none[r] = False
        assert torch.all((self.h.double() - href).abs() <= hoff), float(((self.h.double() - href).abs() - hoff).max())
        off += 2.0 ** -23 * ref.abs()
        tol = off + 2.0 ** -8 * (ref.abs() + off) + 2.0 ** -133
        assert torch.all((y.double() - ref).abs() <= tol), float(((y.double() - ref).abs() / tol).max())
        bits = torch.zeros_like(y) if base is None else base
        assert torch.equal(y[none].view(torch.int16), bits[none].contiguous().view(torch.int16))

    def check_backward(self, dx, da, db, base="own", h=None):
        base = self.dbase if base == "own" else base
        h = self.h if h is None else h
        ref = torch.zeros((self.rows, self.k), dtype=torch.float64, device="cuda") if base is None else base.double()
        off = torch.zeros_like(ref)
        dh = torch.zeros_like(self.dh, dtype=torch.float64)
        dhoff = torch.zeros_like(dh)
        for i, r in enumerate(self.groups()):
            dy, x, s = self.dy[r].double(), self.x[r].double(), float(self.bank.scale[i])
            a, b = self.bank.a[i].double(), self.bank.b[i].double()
            dh[r], dhoff[r] = s * (dy @ b), s * (self.n / 128 + 9) * STEP * (dy.abs() @ b.abs())
            into = dhoff[r] + (2.0 ** -17 + (self.rank / 8 + 2) * STEP) * dh[r].abs()
            ref[r] += dh[r] @ a
            off[r] = into @ a.abs()
            # A gradient's sum over the rows: one step for 16 rows and part, and the tiles' sums.
            sums = (len(r) / 8 + 16) * STEP + 2.0 ** -17
            for got, want, e in ((da, dh[r].t() @ x, (dhoff[r] + sums * dh[r].abs()).t() @ x.abs()),
                                 (db, s * (dy.t() @ h[r].double()), s * (sums + 2.0 ** -23) * (dy.abs().t() @ h[r].double().abs()))):
                if got is not None:
                    tol = e + 2.0 ** -8 * (want.abs() + e) + 2.0 ** -133
                    assert torch.all((got[i].double() - want).abs() <= tol), float(((got[i].double() - want).abs() / tol).max())
        assert torch.all((self.dh.double() - dh).abs() <= dhoff)
        if dx is not None:
            off += 2.0 ** -23 * ref.abs()
            tol = off + 2.0 ** -8 * (ref.abs() + off) + 2.0 ** -133
            assert torch.all((dx.double() - ref).abs() <= tol), float(((dx.double() - ref).abs() / tol).max())

    def like(self):
        e = torch.empty_like
        return (torch.full((self.rows, self.k), 3.0, dtype=BF, device="cuda"), e(self.bank.a).fill_(3.0),
                e(self.bank.b).fill_(3.0))


FEW = [(1, 64, 48, 8, 1), (1, 4096, 1024, 16, 3), (5, 100, 37, 3, 2), (33, 1000, 2000, 64, 5), (64, 257, 130, 128, 7),
       (7, 8, 8, 1, 1), (64, 512, 512, 12, 64), (3, 1, 1, 1, 2), (16, 2048, 72, 32, 4), (2, 33, 5000, 100, 2)]
MANY = [(65, 64, 96, 8, 1), (300, 1600, 801, 16, 5), (777, 160, 4801, 8, 5), (513, 1536, 1024, 64, 8), (200, 96, 33, 128, 3),
        (129, 40, 40, 5, 2), (2100, 768, 512, 16, 2), (500, 72, 1000, 24, 7), (3000, 8, 24, 4, 1), (400, 256, 320, 16, 1024),
        (70, 1, 1, 1, 1), (260, 520, 264, 33, 3), (1500, 300, 1601, 12, 40)]


@pytest.mark.parametrize("kind", ["random", "same", "none", "bad"])
@pytest.mark.parametrize("rows,k,n,rank,count", FEW)
def test_few_rows(rows, k, n, rank, count, kind):
    c = Case(rows, k, n, rank, count, kind)
    y = torch.full((rows, n), 3.0, dtype=BF, device="cuda")
    assert c.forward(y) is y
    c.check_forward(y)
    first = c.h.clone()
    c.forward(y, base=None)
    c.check_forward(y, base=None)
    assert torch.equal(c.h, first)


@pytest.mark.parametrize("kind", ["random", "runs", "same", "none", "bad"])
@pytest.mark.parametrize("rows,k,n,rank,count", MANY)
def test_many_rows(rows, k, n, rank, count, kind):
    c = Case(rows, k, n, rank, count, kind)
    y = torch.full((rows, n), 3.0, dtype=BF, device="cuda")
    c.forward(y)
    c.check_forward(y)
    again = torch.empty_like(y)
    c.forward(again, route=c.q.AdapterRoute(rows, count).set(c.index))
    assert torch.equal(y, again)
    c.forward(again, base=None)
    c.check_forward(again, base=None)


@pytest.mark.parametrize("kind", ["random", "runs", "same", "none", "bad"])
@pytest.mark.parametrize("rows,k,n,rank,count", MANY + FEW[:5])
def test_backward(rows, k, n, rank, count, kind):
    c = Case(rows, k, n, rank, count, kind)
    c.forward(torch.empty((rows, n), dtype=BF, device="cuda"))
    dx, da, db = c.like()
    c.backward(dx, da, db)
    c.check_backward(dx, da, db)
    for i, r in enumerate(c.groups()):
        if len(r) == 0:
            assert not da[i].any() and not db[i].any()
    more = c.like()
    c.backward(*more, route=c.q.AdapterRoute(rows, count).set(c.index))
    assert all(torch.equal(a, b) for a, b in zip((dx, da, db), more))


@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("k,n,rank,shift,pad", [(128, 192, 16, 1, 0), (121, 250, 8, 3, 2), (256, 256, 32, 8, 8),
                                                (64, 1001, 7, 0, 0), (96, 96, 64, 4, 0)])
def test_strided_and_in_place(rows, k, n, rank, shift, pad):
    c = Case(rows, k, n, rank, 4, "random", 7, shift, pad)
    full = torch.full((rows, n + 24), 7.0, dtype=BF, device="cuda")
    y, want = full[:, 3:3 + n], full.clone()
    c.forward(y)
    c.check_forward(y)
    want[:, 3:3 + n] = y
    assert torch.equal(full, want)
    inplace = torch.zeros((rows, n + 5), dtype=BF, device="cuda")[:, :n]
    inplace.copy_(c.base)
    c.forward(inplace, base=inplace)
    assert torch.equal(inplace, y)
    full = torch.full((rows, k + 24), 7.0, dtype=BF, device="cuda")
    dx, want = full[:, 5:5 + k], full.clone()
    _, da, db = c.like()
    c.backward(dx, da, db)
    c.check_backward(dx, da, db)
    want[:, 5:5 + k] = dx
    assert torch.equal(full, want)
    inplace = c.dbase.clone()
    c.backward(inplace, None, None, base=inplace)
    assert torch.equal(inplace, dx)


def test_an_unaligned_bank():
    c = Case(150, 64, 96, 8, 3, "random", 9)
    flat = [torch.zeros(t.numel() + 1, dtype=BF, device="cuda")[1:].view(t.shape) for t in (c.bank.a, c.bank.b)]
    for f, t in zip(flat, (c.bank.a, c.bank.b)):
        f.copy_(t)
    y = torch.empty((150, 96), dtype=BF, device="cuda")
    c.forward(y)
    aligned = c.bank
    c.bank = c.q.Adapters(flat[0], flat[1], aligned.scale)
    again = torch.empty_like(y)
    c.forward(again)
    assert torch.equal(again, y)
    dx, da, db = c.like()
    odd = [torch.zeros(t.numel() + 1, dtype=BF, device="cuda")[1:].view(t.shape) for t in (da, db)]
    c.backward(dx, odd[0], odd[1])
    c.check_backward(dx, odd[0], odd[1])


def test_only_some_gradients():
    c = Case(333, 200, 120, 16, 3, "runs", 11)
    c.forward(torch.empty((333, 120), dtype=BF, device="cuda"))
    whole, (dx, da, db) = c.like(), c.like()
    c.backward(*whole)
    for wanted in ((dx, None, None), (None, da, None), (None, None, db), (dx, None, db)):
        c.backward(*wanted)
        for a, b in zip(wanted, whole):
            assert a is None or torch.equal(a, b)
    c.q.adapter_backward(c.dy, None, None, c.index, c.bank, c.dh, dx, None, None, c.ws)
    c.check_backward(dx, None, None, base=None)


def test_a_small_workspace_gives_the_same_gradients_within_bounds():
    """Without room to lay out the weight gradients' operands they are made where they are used."""
    c = Case(1300, 264, 200, 16, 2, "runs", 13)
    c.forward(torch.empty((1300, 200), dtype=BF, device="cuda"))

    class Small:
        def __init__(self, ws, nbytes):
            self.buf, self.ptr, self.nbytes = ws.buf, ws.ptr, nbytes

    dx, da, db = c.like()
    c.ws = Small(c.ws, 33024 + (1300 + 4) * 4 + 512)
    c.backward(dx, da, db)
    c.check_backward(dx, da, db)
    c.ws = Small(c.ws, 33024)
    with pytest.raises(c.q.Fp8linError):  # no room for the sorted rows
        c.backward(dx, da, db)
    c.backward(dx, da, db, route=c.q.AdapterRoute(1300, 2).set(c.index))
    c.check_backward(dx, da, db)


@pytest.mark.parametrize("rows", [50, 500])
def test_nan_and_infinity_stay_in_their_rows(rows):
    c = Case(rows, 200, 104, 16, 4, "random", 15)
    c.index[:8] = torch.tensor([0, 1, 2, 3, -1, 0, 1, 2], device="cuda")
    y, y2 = (torch.empty((rows, 104), dtype=BF, device="cuda") for _ in range(2))
    c.forward(y)
    clean = c.x.clone()
    c.x[1, 3], c.x[2, 199], c.x[4, 0] = float("nan"), float("inf"), float("nan")  # row 4 has no adapter
    c.forward(y2)
    assert torch.isnan(y2[1]).all() and not torch.isfinite(y2[2]).any()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[1] = keep[2] = False
    assert torch.equal(y[keep], y2[keep])
    # In the backward of these rows: dx keeps to its row, and only these adapters' dA have a NaN.
    c.x.copy_(clean)
    c.forward(y)
    dx, da, db = c.like()
    c.backward(dx, da, db)
    dx2, da2, db2 = c.like()
    c.dy[1, 5] = float("nan")
    c.backward(dx2, da2, db2)
    assert torch.isnan(dx2[1]).all() and torch.isnan(da2[1]).all() and torch.isnan(db2[1][5]).all()
    keep[2] = True
    assert torch.equal(dx[keep], dx2[keep])
    for i in (0, 2, 3):
        assert torch.equal(da[i], da2[i]) and torch.equal(db[i], db2[i])


def test_against_differences():
    """<dx, u>, <dA, v>, <dB, w> against differences of sum(dy y) in 64 bits, which is linear in x and
    bilinear in A and B: central differences are exact but for rounding.  What is left is bf16's
    half step of each value and hi + lo."""
    c = Case(190, 72, 56, 8, 3, "random", 17)
    c.forward(torch.empty((190, 56), dtype=BF, device="cuda"))
    dx, da, db = c.like()
    c.backward(dx, da, db, base=None)
    g = torch.Generator(device="cuda").manual_seed(18)
    x, a, b = c.x.double(), c.bank.a.double(), c.bank.b.double()

    def loss(x, a, b):
        total = 0.0
        for i, r in enumerate(c.groups()):
            total += float((c.dy[r].double() * (x[r] @ a[i].t() @ b[i].t())).sum()) * float(c.bank.scale[i])
        return total

    for got, at in ((dx, 0), (da, 1), (db, 2)):
        u = torch.randn(got.shape, generator=g, device="cuda").double()
        args = [x, a, b]
        up, down = list(args), list(args)
        up[at], down[at] = args[at] + u, args[at] - u
        want = (loss(*up) - loss(*down)) / 2
        terms = got.double() * u
        assert abs(float(terms.sum()) - want) <= (2.0 ** -8 + 2.0 ** -12) * float(terms.abs().sum())


def test_captured_and_replayed_on_another_stream():
    c = Case(260, 192, 160, 16, 3, "runs", 19)
    few = Case(20, 192, 160, 16, 3, "random", 20)
    y, (dx, da, db) = torch.empty((260, 160), dtype=BF, device="cuda"), c.like()
    y2 = torch.empty((20, 160), dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def work():
        c.forward(y)
        c.backward(dx, da, db)
        few.forward(y2)

    with torch.cuda.stream(side):
        work()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            work()
    for seed in (21, 22):  # other rows and other adapters in the same buffers
        c.x.copy_(normal((260, 192), seed))
        c.index.copy_(make_index(260, 3, "random", seed))
        few.index.copy_(make_index(20, 3, "random", seed))
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            graph.replay()
        torch.cuda.synchronize()
        c.check_forward(y)
        c.check_backward(dx, da, db)
        few.check_forward(y2)


def test_offsets_beyond_32_bits():
    import quantised_gemm_gb300 as q
    rows, cols = 70000, 40
    wide = torch.empty((rows, 36000), dtype=BF, device="cuda")  # 5 GB
    c = Case(rows, cols, cols, 8, 3, "random", 23)
    x = wide[:, 35000:35000 + cols]
    x.copy_(c.x)
    y = wide[:, 100:100 + cols]
    y.copy_(c.base)
    c.x = x
    c.forward(y, base=y)
    c.check_forward(y)
    w = torch.ones(cols, dtype=BF, device="cuda")
    a, b = torch.empty_like(c.base), wide[:, 200:200 + cols]
    q.layer_norm(x, w, None, a)
    q.layer_norm(x, w, None, b)
    assert torch.equal(a, b)


def test_no_rows():
    c = Case(0, 64, 32, 8, 2)
    c.forward(torch.empty((0, 32), dtype=BF, device="cuda"))
    _, da, db = c.like()
    c.backward(None, da, db)
    assert not da.any() and not db.any()
    route = c.q.AdapterRoute(0, 2).set(c.index)
    assert route.buf[:4].tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("rows,count,kind", [(1, 1, "same"), (33, 4, "random"), (20000, 1024, "random"), (8193, 1, "same"), (5000, 1024, "random"), (70001, 7, "runs"),
                                             (4096, 3, "none"), (1000, 1000, "bad")])
def test_route(rows, count, kind):
    import quantised_gemm_gb300 as q
    index = make_index(rows, count, kind, 31)
    route = q.AdapterRoute(rows, count).set(index)
    group = torch.where((index >= 0) & (index < count), index, count).long()
    first = torch.zeros(count + 2, dtype=torch.int64, device="cuda")
    first[1:] = torch.bincount(group, minlength=count + 1).cumsum(0)
    assert torch.equal(route.buf[:count + 2].long(), first)
    assert torch.equal(route.buf[count + 2:count + 2 + rows].long(), torch.sort(group, stable=True).indices)


def test_refusals():
    import quantised_gemm_gb300 as q
    c = Case(4, 64, 48, 8, 2)
    y = torch.empty((4, 48), dtype=BF, device="cuda")
    good = dict(x=c.x, index=c.index, bank=c.bank, y=y, h=c.h, ws=c.ws, base=c.base, route=None)
    q.adapter_linear(**good)
    errors = (ValueError, TypeError, q.Fp8linError)
    for change in (dict(x=c.x[:, :63]), dict(x=c.x.float()), dict(index=c.index.long()), dict(index=c.index[:3]), dict(y=y[:3]),
                   dict(h=c.h[:, :7]), dict(h=c.h.double()), dict(ws=None), dict(base=c.base[:, :47]), dict(x=c.x.cpu()),
                   dict(route=q.AdapterRoute(4, 2)), dict(route=q.AdapterRoute(5, 2)), dict(x=c.x.t()),
                   dict(route=q.AdapterRoute(4, 3).set(c.index))):
        with pytest.raises(errors):
            q.adapter_linear(**{**good, **change})
    dx, da, db = c.like()
    good = dict(dy=c.dy, x=c.x, h=c.h, index=c.index, bank=c.bank, dh=c.dh, dx=dx, da=da, db=db, ws=c.ws)
    q.adapter_backward(**good)
    for change in (dict(dy=c.dy[:, :47]), dict(x=None), dict(h=None), dict(da=da[:1]), dict(db=db.float()), dict(dx=dx[:, :8]),
                   dict(dh=c.dh.t()), dict(ws=None), dict(base=dx[:2]), dict(index=c.index.cpu())):
        with pytest.raises(errors):
            q.adapter_backward(**{**good, **change})
    a, b, s = c.bank.a, c.bank.b, c.bank.scale
    for bad in ((a[0], b, s), (a, b[:1], s), (a, b, s.double()), (a, b, s[:1]), (a.float(), b, s), (a[:, :4], b, s),
                (torch.empty((2, 129, 64), dtype=BF, device="cuda"), torch.empty((2, 48, 129), dtype=BF, device="cuda"), s),
                (torch.empty((0, 8, 64), dtype=BF, device="cuda"), torch.empty((0, 48, 8), dtype=BF, device="cuda"), s[:0])):
        with pytest.raises(errors):
            q.Adapters(*bad)
    with pytest.raises(errors):
        q.AdapterRoute(4, 1025)
    with pytest.raises(errors):
        q.AdapterRoute(-1, 2)


def test_a_bank_whose_tensors_moved_is_refused():
    import quantised_gemm_gb300 as q
    c = Case(4, 64, 48, 8, 2)
    y = torch.empty((4, 48), dtype=BF, device="cuda")
    dx, da, db = c.like()
    kept = c.bank.b.data
    c.bank.b.data = kept.clone()
    with pytest.raises(ValueError):
        q.adapter_linear(c.x, c.index, c.bank, y, c.h, c.ws)
    with pytest.raises(ValueError):
        q.adapter_backward(c.dy, c.x, c.h, c.index, c.bank, c.dh, dx, da, db, c.ws)
    c.bank.b.data = kept
    q.adapter_linear(c.x, c.index, c.bank, y, c.h, c.ws)
    with pytest.raises(q.Fp8linError):
        q.adapter_linear(c.x, c.index, q.Adapters(c.bank.a, c.bank.a.transpose(1, 2).contiguous(), c.bank.scale), c.x,
                         c.h, c.ws)  # y is x


UNEVEN = [[96, 328, 0, 3672], [1, 3100, 15], [1040, 1040, 1040], [0, 0, 4100, 0], [2048, 2047, 1], [130, 0, 130, 2, 5000]]


@pytest.mark.parametrize("lengths", UNEVEN, ids=lambda n: "-".join(map(str, n)))
@pytest.mark.parametrize("k,n,rank", [(1300, 1400, 16), (2600, 72, 5), (2600, 2704, 32), (1288, 1400, 64), (700, 901, 128),
                                      (40, 64, 16)])
def test_gradients_of_uneven_adapters(k, n, rank, lengths):
    """Rows that are split evenly whatever an adapter has: one over many CTAs, several in one."""
    count = len(lengths)
    rows = sum(lengths) + 33
    c = Case(rows, k, n, rank, count)
    of = torch.arange(-1, count, dtype=torch.int32, device="cuda")
    index = of.repeat_interleave(torch.tensor([33] + lengths, device="cuda"))
    c.index = index[torch.randperm(rows, generator=torch.Generator(device="cuda").manual_seed(9), device="cuda")]
    c.forward(torch.empty((rows, n), dtype=BF, device="cuda"))
    dx, da, db = c.like()
    c.backward(dx, da, db)
    c.check_backward(dx, da, db)
    more = c.like()
    c.backward(*more)
    assert all(torch.equal(a, b) for a, b in zip((dx, da, db), more))
