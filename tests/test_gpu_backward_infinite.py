"""Backward pass with infinities and NaN in d_out, as an overflowed loss leaves them: every gradient is what the formula gives
over the seen pairs alone (finite, +inf, -inf or NaN), and the call takes about as long as another."""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from plain_backward import NAMES
from test_gpu_backward import SCALE, make, run
from test_gpu_backward_masked import check_rows, expected

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
SHAPES = [([70, 300], [70, 300]), ([64, 1300], [64, 1300]), ([500], [2100]), ([300], [120]), ([1, 129, 255], [3, 131, 400]),
          ([520], [33000])]
IDS = [f"{a}x{b}" for a, b in SHAPES]


def kinds(x):
    return torch.where(torch.isnan(x), 3, torch.where(x == INF, 1, torch.where(x == -INF, 2, 0)))


def dv_kinds(d, b, h):
    """0, 1 (+inf), 2 (-inf) or 3 (NaN) for dv of sequence b and head h: terms p d_out over seen pairs."""
    qs, ks = (slice(int(d[c][b]), int(d[c][b + 1])) for c in ("cu_q", "cu_k"))
    q = torch.cat((d["q_nope"][qs, h], d["q_rope"][qs, h]), -1).double()
    k = torch.cat((d["k_nope"][ks, h], d["k_rope"][ks]), -1).double()
    see = torch.ones((len(q), len(k)), dtype=torch.bool, device=q.device).tril(len(k) - len(q))
    p = torch.exp(SCALE * (q @ k.T) - d["lse"][qs, h].double()[:, None])
    # (unit inputs: no p of a seen pair is below 1e-20, so none rounds to 0)
    assert bool((p[see] > 1e-20).all())
    do, see = d["d_out"][qs, h].double(), see.double()
    up, down, none = (see.T @ m.double() > 0 for m in (do == INF, do == -INF, torch.isnan(do)))
    return torch.where(none | (up & down), 3, torch.where(up, 1, torch.where(down, 2, 0)))


def spoil(d, how, seed):
    x = d["d_out"]
    if how == "column":                    # all rows of every head, and both signs in turn in one
        x[:, :, 3] = INF
        x[::2, 5, 9], x[1::2, 5, 9] = INF, -INF
        return
    g = torch.Generator(device="cuda").manual_seed(seed)
    at = torch.rand(x.shape[:2], generator=g, device="cuda") < 0.02
    e = torch.randint(0, 128, x.shape[:2], generator=g, device="cuda")
    v = torch.tensor([INF, -INF, NAN], device="cuda")[torch.randint(0, 3, x.shape[:2], generator=g, device="cuda")]
    i, h = at.nonzero(as_tuple=True)
    x[i, h, e[i, h]] = v[i, h].to(torch.bfloat16)


@pytest.mark.parametrize("how", ["few", "column"])
@pytest.mark.parametrize("nq,nk", SHAPES, ids=IDS)
def test_gradients_are_the_seen_pairs(cuda_device, nq, nk, how):
    d = make(nq, nk, seed=41 + len(nq))
    spoil(d, how, seed=nk[0])
    got = run(d)
    dv, dk = got[4], got[2]
    exact = expected(d)
    want, bound = exact
    for b in range(len(nq)):
        ks, qs = slice(sum(nk[:b]), sum(nk[:b + 1])), slice(sum(nq[:b]), sum(nq[:b + 1]))
        for h in (0, 5, 64, 127):
            kind = dv_kinds(d, b, h)
            assert torch.equal(kinds(dv[ks, h].double()), kind), (b, h)
            off = (dv[ks, h].double() - want["dv"][ks, h]).abs()
            assert bool(((off <= bound["dv"][ks, h]) | (kind > 0)).all()), (b, h)
            # a key of a head is spoilt in dk by the odd queries that see it, and by no others
            odd = ~torch.isfinite(d["d_out"][qs, h]).all(-1)
            see = torch.ones((nq[b], nk[b]), dtype=torch.bool, device="cuda").tril(nk[b] - nq[b])
            touched = (see & odd[:, None]).any(0)
            assert not bool(torch.isfinite(dk[ks, h][touched].float()).any()), (b, h)
            off = (dk[ks, h].double() - want["dk_nope"][ks, h]).abs()
            assert bool((off <= bound["dk_nope"][ks, h])[~touched].all()), (b, h)
    good = torch.isfinite(d["d_out"]).all(-1).all(-1).nonzero().flatten().tolist()
    check_rows(got, d, NAMES[:2], good, how, exact)
    for x, y in zip(run(d), got):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_an_overflowed_call_takes_about_as_long_as_another(cuda_device):
    n = 4096
    d = make([n], [n], seed=43)
    ws = binding.alloc_workspace_prefill_backward(1, n, n)

    def ms():
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        run(d, workspace=ws)
        start.record()
        run(d, workspace=ws)
        end.record()
        torch.cuda.synchronize()
        return start.elapsed_time(end)

    clean = ms()
    d["d_out"][:, :, 3] = INF
    # (each sum computed again over all its columns: 280 times as long)
    assert ms() < 30 * clean
