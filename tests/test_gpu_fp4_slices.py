"""K slices of a 4-bit product's last tiles where the slices of a tile may not
wait for each other: not every pair with a slice has begun, or other streams'
products hold the SMs.  The same bits as alone, and no time-out."""
import time

import pytest
import torch

import quantised_gemm_gb300 as q

pytestmark = pytest.mark.gpu

# Workspace layout (quantised_gemm_gb300/csrc/internal.h): pairs with a slice begun, done.
SLICES_OFFSET = 224

FORMATS = [q.NVFP4, q.MXFP4]


def operands(M, N, K, fmt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ts, ws = [], q.Workspace()
    for rows in (M, N):
        t = q.Fp4Tensor(rows, K, fmt)
        q.fp4_quantise(torch.randn((rows, K), generator=g, device="cuda").to(torch.bfloat16), t, None, ws)
        ts.append(t)
    return ts


# 100 tiles, the last 24 in three slices; 112, 36 in two; 81, 5 in four.
@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
@pytest.mark.parametrize("M,N,K", [(2500, 2500, 7000), (4096, 1600, 9000), (2200, 2250, 9000)])
def test_slices_that_may_not_wait_leave_all_they_have(M, N, K, fmt):
    a, b = operands(M, N, K, fmt)
    ws = q.Workspace()
    counts = ws.buf[SLICES_OFFSET:SLICES_OFFSET + 8].view(torch.int32)
    # Rows for TMA, and rows without alignment.
    for room in (torch.empty((M, -(-N // 8) * 8), dtype=torch.bfloat16, device="cuda"),
                 torch.empty((M, N + 3), dtype=torch.bfloat16, device="cuda")):
        out = room[:, :N] if room.shape[1] % 8 == 0 else room[:, 1:N + 1]
        q.fp4_gemm(a, b, out, ws)
        want = out.clone()
        assert torch.count_nonzero(counts).item() == 0
        for short in (1, 1000):
            counts[0] = -short               # so many pairs seem not to have begun
            room.fill_(float("nan"))
            torch.cuda.synchronize()
            t0 = time.time()
            q.fp4_gemm(a, b, out, ws)
            q.check(ws)
            assert time.time() - t0 < 1.0
            assert torch.equal(out, want)
            assert torch.count_nonzero(counts).item() == 0
        q.fp4_gemm(a, b, out, ws)
        q.check(ws)
        assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", FORMATS, ids=["nv", "mx"])
def test_split_products_on_two_streams(fmt):
    """Two products whose slices fill the GPU each, on streams of different
    priority, started while a third holds some of the SMs."""
    low, high, side = torch.cuda.Stream(priority=0), torch.cuda.Stream(priority=-1), torch.cuda.Stream()
    sets = [operands(2500, 2500, 7000, fmt, 1), operands(4096, 1600, 9000, fmt, 2)]
    filler = operands(600, 600, 30000, fmt, 3)
    spaces = [q.Workspace() for _ in range(3)]
    want = [q.fp4_gemm(*s, torch.empty((s[0].rows, s[1].rows), dtype=torch.bfloat16, device="cuda"), w)
            for s, w in zip(sets + [filler], spaces)]
    rounds = 20
    outs = [[torch.full_like(want[i], float("nan")) for _ in range(rounds)] for i in range(2)]
    fill = torch.empty_like(want[2])
    torch.cuda.synchronize()
    t0 = time.time()
    for r in range(rounds):
        q.fp4_gemm(*filler, fill, spaces[2], stream=side)
        q.fp4_gemm(*sets[0], outs[0][r], spaces[0], stream=low)
        q.fp4_gemm(*sets[1], outs[1][r], spaces[1], stream=high)
    torch.cuda.synchronize()
    assert time.time() - t0 < 1.0
    for w in spaces:
        q.check(w)
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])
    assert torch.equal(fill, want[2])
