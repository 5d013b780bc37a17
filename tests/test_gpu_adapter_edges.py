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
