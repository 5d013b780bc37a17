"""4-bit quantisation, products and the 4-bit Linear on the GPU against the
64-bit oracle: every code and scale byte equal, values within their type's
rounding, products within the library's GEMM bound."""
import numpy as np
import pytest
import torch

from helpers import assert_within_bound, bf16_to_f64, to_dev_bf16
from oracle import fp4 as o4

pytestmark = pytest.mark.gpu

FORMATS = [o4.NVFP4, o4.MXFP4]
SIZES = [(1, 1), (1, 16), (2, 33), (16, 4096), (31, 15), (33, 47), (127, 64), (128, 128), (129, 65),
         (24, 4096), (25, 3933), (130, 200), (255, 513), (640, 1600), (1009, 1531)]


def make(rows, cols, seed, std=1.0):
    """bf16 bits and their 64-bit values: normal, with large values, blocks of
    zeros and values far below their block's maximum."""
    g = np.random.default_rng(seed)
    x = (g.normal(size=(rows, cols)) * std).astype(np.float32)
    x[g.random((rows, cols)) < 1e-3] *= 40
    x[g.random((rows, cols)) < 1e-2] *= 1e-6
    x[:, : cols // 5] *= (g.random((rows, 1)) < 0.9)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    return bits, (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def dirty(q, rows, cols, fmt, state=None):
    t = q.Fp4Tensor(rows, cols, fmt, state=state)
    t.codes.fill_(0xA5)
    t.scales.fill_(0x5A)
    return t


def check_bytes(t, x, scale, what):
    codes, sc = o4.quantise(x, t.fmt, scale)
    assert np.array_equal(t.codes.cpu().numpy(), o4.pack(codes, x.shape[1])), what + ": codes"
    assert np.array_equal(t.scales.cpu().numpy(), o4.tile_scales(sc)), what + ": scales"


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantise_bytes(rows, cols, fmt):
    import quantised_gemm_gb300 as q
    bits, x = make(rows, cols, rows * 7 + cols)
    xd = to_dev_bf16(bits)
    ws = q.Workspace()
    a = dirty(q, rows, cols, fmt)
    at = dirty(q, cols, rows, fmt, a.state)
    s, inv = o4.tensor_scale(np.abs(x).max())
    q.fp4_quantise(xd, a, at, ws)
    check_bytes(a, x, s, "both")
    check_bytes(at, np.ascontiguousarray(x.T), s, "both, transposed")
    if fmt == o4.NVFP4:
        assert float(a.state.scale) == s and float(a.state.inv_scale) == inv
        assert float(a.state.amax) == np.abs(x).max()
    b = dirty(q, rows, cols, fmt)
    q.fp4_quantise(xd, b, None, ws)
    check_bytes(b, x, s, "out alone")
    bt = dirty(q, cols, rows, fmt)
    q.fp4_quantise(xd, None, bt, ws)
    check_bytes(bt, np.ascontiguousarray(x.T), s, "out_t alone")
    # The values: bf16 is one more rounding, fp32 within the two roundings of its products.
    codes, sc = o4.quantise(x, fmt, s)
    v = o4.values(codes, sc, fmt, cols, inv)
    got = q.fp4_dequantise(a, torch.empty((rows, cols), dtype=torch.float32, device="cuda"))
    assert np.all(np.abs(got.cpu().numpy().astype(np.float64) - v) <= 2.0 ** -23 * np.abs(v))
    got = q.fp4_dequantise(a, torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda"))
    assert np.all(np.abs(bf16_to_f64(got) - v) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(v))
    q.check(ws)


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
@pytest.mark.parametrize("offset,width", [(0, 4), (1, 0), (3, 5), (8, 16)])
def test_strided_rows(fmt, offset, width):
    import quantised_gemm_gb300 as q
    rows, cols = 70, 177
    bits, x = make(rows, cols + offset + width, 11)
    wide = to_dev_bf16(bits)
    x = np.ascontiguousarray(x[:, offset:offset + cols])
    a = dirty(q, rows, cols, fmt)
    at = dirty(q, cols, rows, fmt, a.state)
    ws = q.Workspace()
    q.fp4_quantise(wide[:, offset:offset + cols], a, at, ws)
    s, inv = o4.tensor_scale(np.abs(x).max())
    check_bytes(a, x, s, "strided")
    check_bytes(at, np.ascontiguousarray(x.T), s, "strided, transposed")
    codes, sc = o4.quantise(x, fmt, s)
    v = o4.values(codes, sc, fmt, cols, inv)
    for dtype in (torch.float32, torch.bfloat16):
        room = torch.full((rows, cols + offset + width), 7.0, dtype=dtype, device="cuda")
        q.fp4_dequantise(a, room[:, offset:offset + cols])
        got = room.float().cpu().numpy()
        assert np.all(np.abs(got[:, offset:offset + cols] - v) <= 2.0 ** -7 * np.abs(v))
        assert np.all(got[:, :offset] == 7) and np.all(got[:, offset + cols:] == 7)


@pytest.mark.parametrize("rows,cols", [(5000, 1), (5000, 16), (9001, 17), (2000, 64), (1500, 100), (700, 130),
                                       (600, 256), (601, 257)])
def test_narrow_strided_rows_find_their_largest(rows, cols):
    import quantised_gemm_gb300 as q
    bits, x = make(rows, cols + 16, 12)
    ws = q.Workspace()
    for r, c in ((0, 0), (rows - 1, cols - 1), (rows // 2, cols // 2)):
        y, b = x[:, :cols].copy(), bits.copy()
        y[r, c], b[r, c] = -1000.0, 0xC47A
        b[:, cols:] = 0x7F80                      # beside the rows: infinities
        a = dirty(q, rows, cols, q.NVFP4)
        q.fp4_quantise(to_dev_bf16(b)[:, :cols], a, None, ws)
        assert float(a.state.amax) == 1000.0
        check_bytes(a, y, o4.tensor_scale(1000.0)[0], "narrow")


@pytest.mark.parametrize("algo", ["atomic", "reduction", "precomputed", "single_pass", "auto"])
def test_dynamic_algorithms(algo):
    import quantised_gemm_gb300 as q
    algos = dict(atomic=q.AMAX_ATOMIC, reduction=q.AMAX_REDUCTION, precomputed=q.AMAX_PRECOMPUTED,
                 single_pass=q.AMAX_SINGLE_PASS, auto=q.AMAX_AUTO)
    for rows, cols in ((48, 160), (48, 161), (2048, 512)):
        bits, x = make(rows, cols, 21)
        a = dirty(q, rows, cols, q.NVFP4)
        a.state.amax_algo = algos[algo]
        amax = np.abs(x).max()
        if algo == "precomputed":
            amax *= 2
            a.state.amax.fill_(float(amax))
        q.fp4_quantise(to_dev_bf16(bits), a, None, q.Workspace())
        check_bytes(a, x, o4.tensor_scale(amax)[0], algo)


def test_delayed_scaling():
    import quantised_gemm_gb300 as q
    rows, cols = 65, 130
    st = q.ScalingState(q.E4M3, q.DELAYED, history_len=3)
    a = dirty(q, rows, cols, q.NVFP4, st)
    at = dirty(q, cols, rows, q.NVFP4, st)
    ws = q.Workspace()
    history, scale = [0.0] * 3, None
    for step in range(5):
        bits, x = make(rows, cols, 40 + step, std=1.0 + 3 * step)
        amax = np.abs(x).max()
        if scale is None:
            scale = o4.tensor_scale(amax)[0]  # the first cast takes its own amax
        q.fp4_quantise(to_dev_bf16(bits), a, at, ws)
        check_bytes(a, x, scale, "step %d" % step)
        check_bytes(at, np.ascontiguousarray(x.T), scale, "step %d, transposed" % step)
        assert float(st.amax) == amax and not st.needs_init
        q.scale(st)
        history[step % 3] = amax
        scale = o4.tensor_scale(max(history))[0]
        assert float(st.scale) == scale


@pytest.mark.parametrize("fmt,kind", [(0, "precomputed"), (0, "delayed"), (1, None)])
@pytest.mark.parametrize("rows,cols", [(4100, 2000), (2048, 4096), (8000, 1160)])
def test_many_tiles_equal_few(rows, cols, fmt, kind):
    """A tensor of many tiles against the same rows quantised 384 at a time
    (both held to the oracle at smaller sizes above)."""
    import quantised_gemm_gb300 as q
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((rows, cols), generator=g, device="cuda").to(torch.bfloat16)
    amax = float(x.abs().max())
    ws = q.Workspace()

    def states():
        if fmt == 1:
            return None
        if kind == "delayed":
            st = q.ScalingState(q.E4M3, q.DELAYED, 4)
            st.needs_init = 0
            st.scale.fill_(o4.tensor_scale(amax)[0])
            st.inv_scale.fill_(o4.tensor_scale(amax)[1])
        else:
            st = q.ScalingState(q.E4M3, amax_algo=q.AMAX_PRECOMPUTED)
            st.amax.fill_(amax)
        return st

    def values(part, r):
        st = states()
        a, at = dirty(q, r, cols, fmt, st), dirty(q, cols, r, fmt, st)
        q.fp4_quantise(part, a, at, ws)
        if kind == "delayed":
            assert float(st.amax) == float(part.abs().max())
        return (q.fp4_dequantise(a, torch.empty((r, cols), device="cuda")),
                q.fp4_dequantise(at, torch.empty((cols, r), device="cuda")))

    whole, whole_t = values(x, rows)
    for r0 in range(0, rows, 384):
        r = min(384, rows - r0)
        v, vt = values(x[r0:r0 + r], r)
        assert torch.equal(whole[r0:r0 + r], v) and torch.equal(whole_t[:, r0:r0 + r], vt)
    q.check(ws)


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
def test_large_linear_equals_its_parts(fmt):
    """x and W of many tiles in the forward's one quantisation against two calls."""
    import quantised_gemm_gb300 as q
    M, K, N = 1100, 2048, 3000
    lin = q.Fp4Linear(M, K, N, fmt=fmt)
    x = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    w = (torch.randn((N, K), device="cuda") * 0.02).to(torch.bfloat16)
    lin.forward(x, w)
    ws = q.Workspace()
    for t, tt, src in ((lin.x4, lin.x4t, x), (lin.w4, lin.w4t, w)):
        r, c = src.shape
        a = dirty(q, r, c, fmt)
        at = dirty(q, c, r, fmt, a.state)
        q.fp4_quantise(src, a, at, ws)
        assert torch.equal(a.codes, t.codes) and torch.equal(a.scales, t.scales)
        assert torch.equal(at.codes, tt.codes) and torch.equal(at.scales, tt.scales)
        if a.state is not None:
            for name in ("amax", "scale", "inv_scale"):
                assert torch.equal(getattr(a.state, name), getattr(t.state, name))
    assert torch.equal(lin.y, q.fp4_gemm(lin.x4, lin.w4, torch.empty_like(lin.y), ws))


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nan_and_infinity(fmt, bad):
    import quantised_gemm_gb300 as q
    x = torch.ones((40, 100), dtype=torch.bfloat16, device="cuda")
    x[5, 70] = bad
    a = q.Fp4Tensor(40, 100, fmt)
    at = q.Fp4Tensor(100, 40, fmt, state=a.state)
    q.fp4_quantise(x, a, at, q.Workspace())
    v = q.fp4_dequantise(a, torch.empty((40, 100), device="cuda")).cpu()
    vt = q.fp4_dequantise(at, torch.empty((100, 40), device="cuda")).cpu()
    if fmt == o4.NVFP4:  # the tensorwise scale is gone
        assert torch.isnan(v).all() and torch.isnan(vt).all()
    else:  # only the blocks that hold it
        want = torch.ones(40, 100)
        want[5, 64:96] = float("nan")
        assert torch.equal(torch.isnan(v), torch.isnan(want)) and (v[~torch.isnan(v)] == 1).all()
        want = torch.ones(100, 40)
        want[70, 0:32] = float("nan")
        assert torch.equal(torch.isnan(vt), torch.isnan(want)) and (vt[~torch.isnan(vt)] == 1).all()


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
def test_zeros_subnormals_and_the_largest(fmt):
    import quantised_gemm_gb300 as q
    rows = np.zeros((6, 64), np.uint16)
    rows[1] = 0x8000                       # -0
    rows[2] = 0x0001                       # the smallest subnormal
    rows[3, ::2], rows[3, 1::2] = 0x7F7F, 0xFF7F   # the largest magnitudes
    rows[4] = 0x0080                       # the smallest normal
    rows[5, 0] = 0x3F80
    for sel in ([0, 1], [2, 4], [3], [0, 2, 4, 5], [0, 1, 2, 3, 4, 5]):
        bits = np.ascontiguousarray(rows[sel])
        x = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        a = dirty(q, len(sel), 64, fmt)
        q.fp4_quantise(to_dev_bf16(bits), a, None, q.Workspace())
        check_bytes(a, x, o4.tensor_scale(np.abs(x).max())[0], str(sel))


def test_empty_tensors():
    import quantised_gemm_gb300 as q
    ws = q.Workspace()
    for fmt in FORMATS:
        for rows, cols in ((0, 64), (5, 0), (0, 0)):
            a = q.Fp4Tensor(rows, cols, fmt)
            q.fp4_quantise(torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda"), a, None, ws)
            if a.state is not None:
                assert float(a.state.amax) == 0 and float(a.state.scale) == o4.tensor_scale(0.0)[0]
            q.fp4_dequantise(a, torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda"))
        a, b = q.Fp4Tensor(5, 0, fmt), q.Fp4Tensor(7, 0, fmt)
        for t in (a, b):
            if t.state is not None:
                t.state.inv_scale.fill_(1.0)
        out = torch.full((5, 9), 3.0, dtype=torch.bfloat16, device="cuda")
        q.fp4_gemm(a, b, out[:, :7], ws)   # an empty sum is zero
        assert (out[:, :7] == 0).all() and (out[:, 7:] == 3).all()
        e = q.Fp4Tensor(0, 64, fmt)
        q.fp4_gemm(e, q.Fp4Tensor(7, 64, fmt), torch.empty((0, 7), dtype=torch.bfloat16,
                                                           device="cuda"), ws)


# ---------------------------------------------------------------- products


def quantised(q, rows, cols, fmt, seed, std=1.0):
    """A 4-bit tensor on the device and its exact values without and with the tensorwise factor."""
    bits, x = make(rows, cols, seed, std)
    t = q.Fp4Tensor(rows, cols, fmt)
    q.fp4_quantise(to_dev_bf16(bits), t, None, q.Workspace())
    s, inv = o4.tensor_scale(np.abs(x).max())
    codes, sc = o4.quantise(x, fmt, s)
    return t, o4.values(codes, sc, fmt, cols, inv)


PRODUCTS = [(1, 1, 1), (1, 16, 64), (1, 130, 4096), (2, 257, 100), (16, 128, 256), (17, 96, 31),
            (32, 4096, 1600), (33, 200, 1000), (64, 129, 513), (65, 384, 640), (100, 100, 100),
            (128, 128, 128), (129, 127, 257), (256, 256, 256), (300, 1000, 1531), (777, 333, 96),
            (1024, 512, 4096), (515, 2049, 2048), (70, 200, 6200), (250, 1000, 6144), (129, 130, 9001),
            (2600, 1400, 1000), (2100, 2101, 300), (1300, 4099, 2000)]


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(M, N, K, fmt):
    import quantised_gemm_gb300 as q
    a, va = quantised(q, M, K, fmt, 100 + M)
    b, vb = quantised(q, N, K, fmt, 200 + N, std=0.02)
    ws = q.Workspace()
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    q.fp4_gemm(a, b, out, ws)
    q.check(ws)
    assert_within_bound(bf16_to_f64(out), va @ vb.T, np.abs(va) @ np.abs(vb).T, "fp4 product")
    # Rows with a stride and no alignment: the same bits, and nothing beside them.
    room = torch.full((M, N + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    q.fp4_gemm(a, b, room[:, 1:N + 1], ws)
    assert torch.equal(room[:, 1:N + 1], out)
    assert (room[:, 0] == 5).all() and (room[:, N + 1:] == 5).all()
    # Rows aligned to 16 bytes that end inside 16 bytes.
    room = torch.full((M + 1, -(-N // 8) * 8 + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    q.fp4_gemm(a, b, room[:M, :N], ws)
    assert torch.equal(room[:M, :N], out)
    assert (room[:M, N:] == 5).all() and (room[M] == 5).all()
    again = torch.empty_like(out)
    q.fp4_gemm(a, b, again, ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
@pytest.mark.parametrize("M,N,K", [(2300, 2400, 6000), (4096, 1600, 9000), (2500, 2500, 7000),
                                   (1030, 1400, 8192), (2049, 513, 20000)])
def test_product_split_over_its_last_wave(M, N, K, fmt):
    """Long K loops whose last tiles run as slices: the same as a workspace
    without room for partials gives, within the bound, and the same bits again."""
    import quantised_gemm_gb300 as q
    from quantised_gemm_gb300 import _lib
    g = torch.Generator(device="cuda").manual_seed(M)

    def one(rows, std):
        t = q.Fp4Tensor(rows, K, fmt)
        q.fp4_quantise((torch.randn((rows, K), generator=g, device="cuda") * std).to(torch.bfloat16), t,
                       None, q.Workspace())
        return t, q.fp4_dequantise(t, torch.empty((rows, K), device="cuda"))

    (a, va), (b, vb) = one(M, 1.0), one(N, 0.02)
    ws = q.Workspace()
    out = q.fp4_gemm(a, b, torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), ws)
    q.check(ws)
    ref = (va.double() @ vb.double().t()).cpu().numpy()
    s = (va.abs().double() @ vb.abs().double().t()).cpu().numpy()
    assert_within_bound(bf16_to_f64(out), ref, s, "split product")
    for _ in range(3):
        assert torch.equal(q.fp4_gemm(a, b, torch.empty_like(out), ws), out)
    room = torch.full((M, N + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    q.fp4_gemm(a, b, room[:, 1:N + 1], ws)
    assert (room[:, 0] == 5).all() and (room[:, N + 1:] == 5).all()
    assert_within_bound(bf16_to_f64(room[:, 1:N + 1]), ref, s, "split product, unaligned rows")
    whole = torch.empty_like(out)
    st = q.library().fp8lin_fp4_gemm(a._ref, b._ref, whole.data_ptr(), N, ws.ptr, 32768, q._stream())
    assert st == _lib.OK
    assert_within_bound(bf16_to_f64(whole), ref, s, "whole product")
    q.check(ws)


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
def test_product_of_small_whole_numbers_is_exact(fmt):
    # Values 0, +-1, +-2 in blocks whose maximum is 2: a product of whole numbers below 2^8.
    import quantised_gemm_gb300 as q
    g = np.random.default_rng(8)
    M, N, K = 150, 140, 48
    xs = []
    for rows in (M, N):
        x = g.integers(-2, 3, (rows, K)).astype(np.float32)
        x[:, ::16] = 2
        xs.append(x)
    ts = []
    for x in xs:
        t = q.Fp4Tensor(x.shape[0], K, fmt)
        if t.state is not None:
            t.state.amax_algo = q.AMAX_PRECOMPUTED
            t.state.amax.fill_(2 * 448.0 / 384.0)  # S = 192: c = 384 stands for 2, 6 is 2's code
        q.fp4_quantise(torch.from_numpy(x).to(torch.bfloat16).cuda(), t, None, q.Workspace())
        ts.append(t)
    vals = [q.fp4_dequantise(t, torch.empty(t.rows, K, device="cuda")).cpu().numpy().astype(np.float64)
            for t in ts]
    out = q.fp4_gemm(ts[0], ts[1], torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), q.Workspace())
    ref = vals[0] @ vals[1].T
    assert_within_bound(bf16_to_f64(out), ref, np.abs(vals[0]) @ np.abs(vals[1]).T, "whole numbers")


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
def test_nan_reaches_its_row_only(fmt):
    import quantised_gemm_gb300 as q
    a, va = quantised(q, 200, 320, fmt, 5)
    b, vb = quantised(q, 150, 320, fmt, 6)
    sc = a.scales.view(-1, 512)
    sc[0, (40 % 32) * 16 + (40 // 32) * 4 + 1] = 0x7F if fmt == o4.NVFP4 else 0xFF  # row 40, block 1
    out = q.fp4_gemm(a, b, torch.empty((200, 150), dtype=torch.bfloat16, device="cuda"), q.Workspace())
    nan = torch.isnan(out).cpu()
    assert nan[40].all() and nan.sum() == 150


@pytest.mark.parametrize("fmt,kind", [(0, "dynamic"), (0, "precomputed"), (0, "delayed"), (1, None)])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 257, 4096), (2, 128, 100), (3, 5000, 300), (8, 96, 2048),
                                   (1, 9000, 14336), (16, 130, 1000), (17, 640, 513), (32, 4096, 4096),
                                   (32, 33, 31), (5, 40000, 512)])
def test_linear_of_few_tokens_equals_its_parts(M, N, K, fmt, kind):
    """One launch: the quantised tokens, their state and y are those of the
    quantisation and the product by themselves, bit for bit."""
    import quantised_gemm_gb300 as q
    bits, x = make(M, K, 60 + M)
    xd = to_dev_bf16(bits)
    w = q.Fp4Tensor(N, K, fmt)
    g = torch.Generator(device="cuda").manual_seed(70)
    q.fp4_quantise((torch.randn((N, K), generator=g, device="cuda") * 0.02).to(torch.bfloat16), w, None,
                   q.Workspace())
    amax = np.abs(x).max()

    def tokens():
        st = None
        if fmt == 0:
            st = q.ScalingState(q.E4M3, q.DELAYED if kind == "delayed" else q.DYNAMIC, 2,
                                q.AMAX_PRECOMPUTED if kind == "precomputed" else q.AMAX_AUTO)
            st.amax.fill_(float(amax) if kind == "precomputed" else 9e9)
        return dirty(q, M, K, fmt, st)

    for step in range(2 if kind == "delayed" else 1):  # the first delayed call takes its own amax
        a, b = (tokens(), tokens()) if step == 0 else (a, b)
        ws = q.Workspace()
        y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        q.fp4_linear(xd, a, w, y, ws)
        q.check(ws)
        q.fp4_quantise(xd, b, None, ws)
        want = q.fp4_gemm(b, w, torch.empty_like(y), ws)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
        if a.state is not None:
            assert a.state.needs_init == 0
            for name in ("amax", "scale", "inv_scale"):
                assert torch.equal(getattr(a.state, name), getattr(b.state, name)), name
        assert torch.equal(y, want)
        xd = xd * 2
    if K > 8:  # tokens with a stride, y's rows unaligned
        wide = torch.zeros((M, K + 5), dtype=torch.bfloat16, device="cuda")
        wide[:, 3:3 + K] = to_dev_bf16(bits)
        room = torch.full((M, N + 3), 5.0, dtype=torch.bfloat16, device="cuda")
        c = tokens()
        q.fp4_linear(wide[:, 3:3 + K], c, w, room[:, 1:N + 1], q.Workspace())
        d = tokens()
        q.fp4_quantise(to_dev_bf16(bits), d, None, ws)
        assert torch.equal(c.codes, d.codes) and torch.equal(c.scales, d.scales)
        assert torch.equal(room[:, 1:N + 1], q.fp4_gemm(d, w, torch.empty_like(y), ws))
        assert (room[:, 0] == 5).all() and (room[:, N + 1:] == 5).all()


@pytest.mark.parametrize("M", [1, 16, 200])
def test_product_on_another_stream(M):
    import quantised_gemm_gb300 as q
    bits, x = make(M, 512, 9)
    w, vw = quantised(q, 256, 512, o4.NVFP4, 10)
    x4, ws = q.Fp4Tensor(M, 512, o4.NVFP4), q.Workspace()
    xd = to_dev_bf16(bits)
    y0 = torch.empty((M, 256), dtype=torch.bfloat16, device="cuda")
    q.fp4_linear(xd, x4, w, y0, ws)
    torch.cuda.synchronize()
    y1 = torch.empty_like(y0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        src = xd.clone()
        q.fp4_linear(src, x4, w, y1, ws)
    side.synchronize()
    assert torch.equal(y0, y1)


def test_linear_in_a_graph():
    import quantised_gemm_gb300 as q
    w, vw = quantised(q, 320, 640, o4.NVFP4, 12)
    x4, ws = q.Fp4Tensor(4, 640, o4.NVFP4), q.Workspace()
    x = torch.zeros((4, 640), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((4, 320), dtype=torch.bfloat16, device="cuda")
    q.fp4_linear(x, x4, w, y, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.fp4_linear(x, x4, w, y, ws)
    for seed in (1, 2):
        bits, xv = make(4, 640, seed)
        x.copy_(to_dev_bf16(bits))
        g.replay()
        want = torch.empty_like(y)
        q.fp4_linear(x, q.Fp4Tensor(4, 640, o4.NVFP4), w, want, q.Workspace())
        assert torch.equal(y, want)


# ---------------------------------------------------------------- the Linear


@pytest.mark.parametrize("fmt,scaling", [(0, "dynamic"), (0, "delayed"), (1, "dynamic")])
@pytest.mark.parametrize("M,K,N", [(1, 64, 48), (48, 160, 96), (130, 257, 131), (256, 512, 384)])
def test_linear_forward_backward(M, K, N, fmt, scaling):
    import quantised_gemm_gb300 as q
    lin = q.Fp4Linear(M, K, N, fmt=fmt, scaling=scaling)
    xb, x = make(M, K, 1)
    wb, w = make(N, K, 2, std=0.05)
    db, dy = make(M, N, 3, std=1e-3)
    y = lin.forward(to_dev_bf16(xb), to_dev_bf16(wb))
    dx, dw = lin.backward(to_dev_bf16(db))
    q.check(lin.ws)

    def val(v):
        s, inv = o4.tensor_scale(np.abs(v).max())

        def one(m):
            c, sc = o4.quantise(np.ascontiguousarray(m), fmt, s)
            return o4.values(c, sc, fmt, m.shape[1], inv)
        return one(v), one(v.T)

    (x4, x4t), (w4, w4t), (d4, d4t) = val(x), val(w), val(dy)
    for got, a, b, what in ((y, x4, w4, "y"), (dx, d4, w4t, "dX"), (dw, d4t, x4t, "dW")):
        assert_within_bound(bf16_to_f64(got), a @ b.T, np.abs(a) @ np.abs(b).T, what)
    lin.sync_scales()
    only = lin.backward(to_dev_bf16(db), need_dw=False)
    assert only[1] is None and (scaling == "delayed" or torch.equal(only[0], dx))


def test_kept_weight():
    import quantised_gemm_gb300 as q
    lin = q.Fp4Linear(32, 128, 64)
    xb, _ = make(32, 128, 1)
    wb, _ = make(64, 128, 2)
    x, w = to_dev_bf16(xb), to_dev_bf16(wb)
    with pytest.raises(ValueError):
        lin.forward(x, None)                   # no weight yet
    y = lin.forward(x, w).clone()
    kept = lin.w4.codes.clone()
    lin.w4.codes.zero_()
    assert (lin.forward(x, None) == 0).all()   # the weight's 4-bit copy is used as it is
    lin.w4.codes.copy_(kept)
    assert torch.equal(lin.forward(x, None), y)
    lin.w4.codes.zero_()
    assert torch.equal(lin.forward(x, w * 2.0), y * 2)  # a weight that is given is quantised
    lin = q.Fp4Linear(32, 128, 64, scaling="delayed")
    lin.step(x, w, x[:, :64].contiguous())
    with pytest.raises(ValueError):
        lin.forward(x, None)                   # its scale has moved on
    lin.forward(x, w)
    lin.forward(x, None)


def test_python_refusals():
    import quantised_gemm_gb300 as q
    ws = q.Workspace()
    x = torch.zeros((16, 32), dtype=torch.bfloat16, device="cuda")
    a = q.Fp4Tensor(16, 32)
    with pytest.raises(TypeError):
        q.fp4_quantise(x.float(), a, None, ws)
    with pytest.raises(ValueError):
        q.fp4_quantise(x.cpu(), a, None, ws)
    with pytest.raises(ValueError):
        q.fp4_quantise(x.t(), q.Fp4Tensor(32, 16), None, ws)       # columns not contiguous
    with pytest.raises(ValueError):
        q.fp4_quantise(x, None, None, ws)
    with pytest.raises(ValueError):
        q.fp4_quantise(x, a, q.Fp4Tensor(32, 16), ws)              # two states
    with pytest.raises(q.Fp8linError):
        q.fp4_quantise(x, q.Fp4Tensor(16, 48), None, ws)
    with pytest.raises(ValueError):
        q.fp4_gemm(a, q.Fp4Tensor(8, 32), torch.empty((16, 9), dtype=torch.bfloat16, device="cuda"), ws)
    with pytest.raises(q.Fp8linError):
        q.fp4_gemm(a, q.Fp4Tensor(8, 32, q.MXFP4),
                   torch.empty((16, 8), dtype=torch.bfloat16, device="cuda"), ws)
    with pytest.raises(ValueError):
        q.Fp4Tensor(16, 32, q.MXFP4, state=a.state)
    with pytest.raises(ValueError):
        q.Fp4Tensor(16, 32, codes=torch.zeros((16, 8), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        q.Fp4Linear(16, 16, 16, fmt=q.MXFP4, scaling="delayed")
    with pytest.raises(ValueError):
        q.Fp4Linear(16, 32, 16).forward(x[:8], torch.zeros((16, 32), dtype=torch.bfloat16,
                                                           device="cuda"))


# Rows and columns, columns beside them, values before the first, launches.
@pytest.mark.parametrize("rows,cols,beside,before,launches", [
    (16, 4096, 0, 0, 1), (24, 4096, 0, 0, 1), (1, 32768, 0, 0, 1), (128, 256, 8, 0, 1), (100, 100, 1, 0, 1),
    (2048, 1, 7, 0, 1), (1, 98304, 0, 0, 2), (98304, 1, 0, 0, 2), (98304, 1, 7, 0, 2), (4, 24576, 0, 0, 2),
    (310, 310, 1, 0, 2), (16, 4096, 8, 0, 2), (24, 4095, 0, 1, 2), (5000, 1, 7, 0, 2), (2049, 1, 7, 0, 2)])
def test_one_launch_where_scanning_the_tensor_is_cheap(rows, cols, beside, before, launches):
    """Every tile's CTA of the one-launch form scans the whole tensor, so its
    cost is the scan's loads times the tiles, not the values."""
    import quantised_gemm_gb300 as q
    bits, x = make(rows, cols + beside, 31)
    x = np.ascontiguousarray(x[:, :cols])
    room = torch.zeros(before + bits.size, dtype=torch.bfloat16, device="cuda")
    room[before:] = to_dev_bf16(bits).view(-1)
    xd = room[before:].view(rows, cols + beside)[:, :cols]
    a, ws = dirty(q, rows, cols, q.NVFP4), q.Workspace()
    n0 = q.launch_count()
    q.fp4_quantise(xd, a, None, ws)
    assert q.launch_count() - n0 == launches
    check_bytes(a, x, o4.tensor_scale(np.abs(x).max())[0], "bytes")
    assert float(a.state.amax) == np.abs(x).max()


@pytest.mark.parametrize("kind", ["delayed", "precomputed"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nan_and_infinity_at_a_stored_scale(bad, kind):
    """A NaN takes its block with it, an infinity saturates, the rest stays;
    the recorded amax shows both (fp8lin_scale leaves open what it makes of a
    NaN; an infinity leaves no scale)."""
    import quantised_gemm_gb300 as q
    rows, cols = 40, 100
    s, inv = o4.tensor_scale(1.0)
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[5, 70] = bad
    st = q.ScalingState(q.E4M3, q.DELAYED, 1) if kind == "delayed" else \
        q.ScalingState(q.E4M3, amax_algo=q.AMAX_PRECOMPUTED)
    st.needs_init = 0
    st.amax.fill_(1.0), st.scale.fill_(s), st.inv_scale.fill_(inv)
    a, at = q.Fp4Tensor(rows, cols, state=st), q.Fp4Tensor(cols, rows, state=st)
    ws = q.Workspace()
    q.fp4_quantise(x, a, at, ws)
    one = np.float32(6 * 448) * (np.float32(inv) / np.float32(6))   # 1 and the largest value alike
    for t, (r, c), width in ((a, (5, 70), 64), (at, (70, 5), 0)):
        v = q.fp4_dequantise(t, torch.empty((t.rows, t.cols), device="cuda")).cpu()
        want = torch.full(v.shape, float(one))
        if bad == bad:
            want[r, c] = float(one) * (1 if bad > 0 else -1)
        else:
            want[r, width:width + 16] = bad
        assert torch.equal(torch.nan_to_num(v, nan=7.0), torch.nan_to_num(want, nan=7.0))
    if kind == "delayed":
        assert torch.equal(torch.nan_to_num(st.amax.cpu(), 7.0), torch.nan_to_num(torch.tensor([abs(bad)]), 7.0))
        if bad == bad:
            q.scale(st)
            b = q.Fp4Tensor(rows, cols, state=st)
            q.fp4_quantise(torch.ones_like(x), b, None, ws)
            assert torch.isnan(q.fp4_dequantise(b, torch.empty((rows, cols), device="cuda"))).all()
    # Few tokens: quantised in the product's launch, the same bytes and products.
    w, _ = quantised(q, 130, cols, q.NVFP4, 3)
    st.amax.fill_(1.0), st.scale.fill_(s), st.inv_scale.fill_(inv)
    few, part = q.Fp4Tensor(8, cols, state=st), q.Fp4Tensor(8, cols, state=st)
    y = q.fp4_linear(x[:8], few, w, torch.empty((8, 130), dtype=torch.bfloat16, device="cuda"), ws)
    st.amax.fill_(1.0)
    q.fp4_quantise(x[:8], part, None, ws)
    assert torch.equal(few.codes, part.codes) and torch.equal(few.scales, part.scales)
    want = q.fp4_gemm(part, w, torch.empty_like(y), ws)
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(y.nan_to_num(), want.nan_to_num())
    assert torch.isnan(y[5]).all() == (bad != bad) and not torch.isnan(y[:5]).any()


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
@pytest.mark.parametrize("M,N,K", [(1, 100, 300), (20, 200, 500), (130, 257, 513), (1300, 1500, 700)])
def test_codes_with_a_longer_row_stride(M, N, K, fmt):
    import quantised_gemm_gb300 as q
    ws = q.Workspace()

    def pair(rows, cols, state=None):
        """A tensor in wider rows of codes, and the whole rows."""
        ld = -(-cols // 32) * 16
        room = torch.full((rows, ld + 48), 0xA5, dtype=torch.uint8, device="cuda")
        t = q.Fp4Tensor(rows, cols, fmt, state=state, codes=room[:, 16:16 + ld])
        return t, (room[:, :16], room[:, 16 + ld:])

    dense, wide = {}, {}
    for name, rows, std in (("a", M, 1.0), ("b", N, 0.05)):
        bits, x = make(rows, K, 80 + rows, std)
        t, sides = pair(rows, K)
        tt, sides_t = pair(K, rows, t.state)
        q.fp4_quantise(to_dev_bf16(bits), t, tt, ws)
        s, _ = o4.tensor_scale(np.abs(x).max())
        check_bytes(t, x, s, name)
        check_bytes(tt, np.ascontiguousarray(x.T), s, name + ", transposed")
        assert all((p == 0xA5).all() for p in sides + sides_t)
        d = dirty(q, rows, K, fmt)
        q.fp4_quantise(to_dev_bf16(bits), d, None, ws)
        for dtype in (torch.float32, torch.bfloat16):
            v, w = (q.fp4_dequantise(i, torch.empty((rows, K), dtype=dtype, device="cuda")) for i in (t, d))
            assert torch.equal(v, w)
        wide[name], dense[name] = t, d
        if name == "a":
            xd = to_dev_bf16(bits)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    want = q.fp4_gemm(dense["a"], dense["b"], out, ws).clone()
    assert torch.equal(q.fp4_gemm(wide["a"], wide["b"], out, ws), want)
    x4, sides = pair(M, K)
    assert torch.equal(q.fp4_linear(xd, x4, wide["b"], out, ws), want)
    assert torch.equal(x4.codes, dense["a"].codes) and all((p == 0xA5).all() for p in sides)
    q.check(ws)
