"""A bounded wait of the 4-bit products that runs out is reported, not hung
on, and the workspace recovers.  The failure is planted on the host as in
test_gpu_failure.py: the counters on which the K slices of the last wave's
tiles wait for each other start so far below zero that the slices can never
all check in.  Every load and MMA has completed before that wait."""
import time

import pytest
import torch

import quantised_gemm_gb300 as q
from quantised_gemm_gb300 import _lib as L

pytestmark = pytest.mark.gpu

# Workspace layout (quantised_gemm_gb300/csrc/internal.h).
TICKETS_OFFSET = 16640
TICKETS = 4096


def test_slices_that_never_meet():
    M, N, K = 2500, 2500, 7000   # 100 tiles: 24 in the last wave, three slices each
    ws = q.Workspace()
    ts = []
    for rows in (M, N):
        t = q.Fp4Tensor(rows, K)
        q.fp4_quantise(torch.randn((rows, K), device="cuda").to(torch.bfloat16), t, None, ws)
        ts.append(t)
    want = q.fp4_gemm(*ts, torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), ws)
    q.check(ws)
    tickets = ws.buf[TICKETS_OFFSET:TICKETS_OFFSET + 4 * TICKETS]
    assert torch.count_nonzero(tickets).item() == 0
    tickets.view(torch.int32).fill_(-(1 << 30))
    t0 = time.time()
    out = torch.empty_like(want)
    q.fp4_gemm(*ts, out, ws)
    with pytest.raises(q.Fp8linError) as ei:
        q.check(ws)
    assert ei.value.status == L.ETIMEOUT
    assert 1.0 < time.time() - t0 < 60.0        # the 2 s limit, not a hang
    assert torch.count_nonzero(tickets).item() == 0
    assert torch.equal(q.fp4_gemm(*ts, out, ws), want)
    q.check(ws)
