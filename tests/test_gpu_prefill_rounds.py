"""Prefill where tiles are about as long and the last round of work items would
leave most SMs idle: its items go out in halves (tiles of 100 to 256 rows, on
152 SMs 4 to 6 of them a head), and where lengths differ (the last heads are
taken together).  Bounds as in the other prefill tests."""
import pytest

from test_gpu_prefill import check, cuda, make, status_run

pytestmark = pytest.mark.gpu

HEADS = [0, 57, 90, 113, 114, 115, 126, 127]


@pytest.mark.parametrize("nq,nk", [([200, 256, 130, 100], [600, 601, 640, 599]), ([1024], [3000]),
                                   ([513, 40, 90], [700, 650, 660]), ([129, 128, 1, 256], [400, 400, 400, 400]),
                                   ([250] * 6, [333] * 6)])
@pytest.mark.parametrize("causal", [True, False])
def test_last_round_in_halves(cuda_device, nq, nk, causal):
    d = make(nq, nk, sum(nq) + sum(nk))
    out, lse = status_run(cuda(d), causal)
    check(out, lse, d, causal, HEADS)


@pytest.mark.parametrize("nq,nk", [([1500], [1500]), ([700, 30, 256], [700, 30, 2000]), ([90] * 9 + [600], [90] * 9 + [1100])])
def test_lengths_that_differ(cuda_device, nq, nk):
    d = make(nq, nk, sum(nq) + sum(nk))
    out, lse = status_run(cuda(d), True)
    check(out, lse, d, True, HEADS)
