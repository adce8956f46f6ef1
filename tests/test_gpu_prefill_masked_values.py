"""Prefill over keys whose values are not finite: a query that does not see such a
key has the bits of the call without it, one that does has what the sum is, and
another column is never touched.  The keys lie before, in and behind the tiles
that the causal mask cuts, in rows of either half of an item."""
import numpy as np
import pytest
import torch

from test_gpu_prefill import cuda, make, status_run

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def expected(d, causal, bad):
    """[nq, 128, 128]: what the bad values make of each result, 0 for the finite ones."""
    nq = d["q_nope"].shape[0]
    ups, downs, nans = (np.zeros((nq, 128, 128), dtype=bool) for _ in range(3))
    cq, ck = d["cu_q"].tolist(), d["cu_k"].tolist()
    for b in range(len(cq) - 1):
        n_q, n_k = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        for key, head, column, value in bad:
            if not ck[b] <= key < ck[b + 1]:
                continue
            # query i sees key j when j <= i + n_k - n_q
            first = max(0, key - ck[b] - (n_k - n_q)) if causal else 0
            kind = nans if value != value else ups if value > 0 else downs
            kind[cq[b] + first:cq[b + 1], head, column] = True
    out = np.zeros((nq, 128, 128))
    out[ups], out[downs] = INF, -INF
    out[nans | (ups & downs)] = NAN
    return out


def check(nq, nk, bad, causal, seed):
    d = make(nq, nk, seed)
    want, wl = status_run(cuda(d), causal)
    for key, head, column, value in bad:
        d["v"][key, head, column] = value
    got, gl = status_run(cuda(d), causal)
    e = torch.from_numpy(expected(d, causal, bad)).cuda()
    finite = e == 0
    assert torch.equal(gl, wl)
    assert torch.equal(got[finite], want[finite])
    g, e = got[~finite].double(), e[~finite]
    # the sum is not finite either way; where one kind of infinity goes in, a
    # weight below bf16's range may leave NaN in its place (a whole tile's keys)
    assert bool((torch.isnan(g) | (g == e)).all())
    return got, e


def spread(nk_total, seed, n):
    rng = np.random.default_rng(seed)
    at = {(int(rng.integers(nk_total)), int(rng.integers(128)), int(rng.integers(128))): (INF, -INF, NAN)[int(rng.integers(3))]
          for _ in range(n)}
    return [k + (v,) for k, v in at.items()]


@pytest.mark.parametrize("nq,nk", [([1], [1]), ([2], [2]), ([40], [40]), ([129, 128, 1], [129, 300, 90]), ([300], [300]),
                                   ([513, 40, 90], [700, 650, 660]), ([140, 3], [20, 5]), ([700], [700]),
                                   ([250] * 6, [333] * 6), ([33] * 40, [33 + i for i in range(40)])])
@pytest.mark.parametrize("causal", [True, False])
def test_only_the_queries_that_see_them(cuda_device, nq, nk, causal):
    for s in range(3):
        check(nq, nk, spread(sum(nk), s, (1, 20, 400)[s]), causal, 3 + s)


@pytest.mark.parametrize("key", [0, 1, 63, 79, 80, 81, 127, 128, 159, 160, 255, 256, 319, 320, 399])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_one_key_of_all_heads(cuda_device, key, value):
    bad = [(key, h, (5 * h + key) % 128, value) for h in range(128)]
    got, _ = check([400], [400], bad, True, 9)
    # the one that sees it first: its own weight is the largest kept in bf16, so the kind is kept
    row = got[key, torch.arange(128), torch.tensor([c for _, _, c, _ in bad])].float().cpu()
    assert bool((torch.isnan(row) if value != value else row == value).all())


def test_both_infinities_give_nan(cuda_device):
    bad = [(100, h, 7, INF) for h in range(128)] + [(130, h, 7, -INF) for h in range(128)]
    got, _ = check([200], [200], bad, True, 11)
    assert bool((got[100:130, :, 7] == INF).all()) and bool(torch.isnan(got[130:, :, 7]).all())


def test_a_whole_sequence_of_nan_beside_finite_ones(cuda_device):
    d = make([100, 60, 300], [100, 60, 400], 12)
    want, wl = status_run(cuda(d))
    d["v"][100:160] = NAN
    d["v"][160 + 399] = NAN                       # the last sequence's last key: its last query alone sees it
    got, gl = status_run(cuda(d))
    keep = [i for i in range(459) if not 100 <= i < 160]
    assert torch.equal(got[keep], want[keep]) and torch.equal(gl, wl)
    assert torch.isnan(got[100:160]).all() and torch.isnan(got[459]).all()
