"""Backward pass: what masked rows hold does not matter, infinities and NaN included; long sequences on both query forms."""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from plain_backward import NAMES, backward, check
from test_gpu_backward import SCALE, make, run

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# (sequences, bad rows of the last sequence): tiles of 128 and of 256 queries
SHAPES = [([70, 300], [70, 300], [299, 260, 140, 1]), ([64, 1300], [64, 1300], [1299, 1290, 700, 255]),
          ([500], [2100], [499, 300, 128, 0]), ([300], [120], [299, 200, 182])]


def expected(d):
    """Gradients and bounds from 64 bits of the same inputs with zeros where they are not finite."""
    clean = {k: (torch.where(torch.isfinite(x), x, torch.zeros_like(x)) if x.is_floating_point() else x) for k, x in d.items()}
    return backward(clean, True, SCALE)


def check_rows(got, d, names, rows, what, exact=None):
    want, bound = exact or expected(d)
    for name, x in zip(NAMES, got):
        if name not in names:
            continue
        off, b = (x.double() - want[name])[rows].abs(), bound[name][rows]
        ok = (off <= b) | ((want[name][rows] == 0) & (x[rows].double() == 0))
        assert bool(ok.all()), (what, name, ok.logical_not().nonzero()[:4].tolist())


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("key", ["k_nope", "k_rope", "v"])
@pytest.mark.parametrize("nq,nk,bad", SHAPES[:3], ids=["300", "1300", "500 of 2100"])
def test_keys_that_queries_do_not_see(cuda_device, nq, nk, bad, key, value):
    d = make(nq, nk, seed=21)
    at = nk[-1] - nq[-1] + bad[0]                      # the last key: the last query alone sees it
    for b in bad[:2]:
        j = sum(nk[:-1]) + nk[-1] - nq[-1] + b
        d[key][(j, 5, 9) if key != "k_rope" else (j, 9)] = value
        at = min(at, nk[-1] - nq[-1] + b)
    d["out"], d["lse"] = binding.mla_prefill_bf16(d["q_nope"], d["q_rope"], d["k_nope"], d["k_rope"], d["v"], d["cu_q"],
                                                  d["cu_k"], SCALE)
    got = run(d)
    first = sum(nq[:-1])
    rows = list(range(first)) + list(range(first, first + at - (nk[-1] - nq[-1])))
    check_rows(got, d, ("dq_nope", "dq_rope"), rows, (key, value))
    # the other sequences' keys
    check_rows(got, d, ("dk_nope", "dk_rope", "dv"), list(range(sum(nk[:-1]))), (key, value))
    # a head's rows alone are spoilt where the value is a head's
    if key != "k_rope":
        other = [h for h in range(128) if h != 5]
        want, bound = expected(d)
        for name, x in zip(NAMES, got):
            if name != "dk_rope":
                assert bool(((x.double() - want[name]).abs() <= bound[name] + 1e-30)[:, other].all()), name


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("key", ["q_nope", "q_rope", "d_out"])
@pytest.mark.parametrize("nq,nk,bad", SHAPES, ids=["300", "1300", "500 of 2100", "300 over 120"])
def test_queries_that_keys_are_not_seen_by(cuda_device, nq, nk, bad, key, value):
    d = make(nq, nk, seed=22)
    off = nk[-1] - nq[-1]
    low = bad[-1] if off >= 0 else bad[1]              # (rows below it are left good)
    i = sum(nq[:-1]) + low
    d[key][i, 77, 3] = value
    d["out"], d["lse"] = binding.mla_prefill_bf16(d["q_nope"], d["q_rope"], d["k_nope"], d["k_rope"], d["v"], d["cu_q"],
                                                  d["cu_k"], SCALE)
    got = run(d)
    keys = list(range(sum(nk[:-1]))) + list(range(sum(nk[:-1]) + max(0, low + off + 1), sum(nk)))
    check_rows(got, d, ("dk_nope", "dk_rope", "dv"), keys, (key, value))
    check_rows(got, d, ("dq_nope", "dq_rope"), [r for r in range(sum(nq)) if r != i], (key, value))


def test_queries_that_see_nothing_hold_anything(cuda_device):
    d = make([300, 40], [120, 40], seed=23)
    for k in ("q_nope", "q_rope", "d_out"):
        d[k][:180] = NAN
    d["out"], d["lse"] = binding.mla_prefill_bf16(d["q_nope"], d["q_rope"], d["k_nope"], d["k_rope"], d["v"], d["cu_q"],
                                                  d["cu_k"], SCALE)
    got = run(d)
    assert not got[0][:180].any() and not got[1][:180].any()
    check_rows(got, d, NAMES[:2], list(range(180, 340)), "dq")
    check_rows(got, d, NAMES[2:], list(range(160)), "dk")


def test_all_of_a_sequence_not_finite(cuda_device):
    d = make([200, 300], [200, 300], seed=24)
    for k in ("q_nope", "q_rope", "d_out", "k_nope", "k_rope", "v"):
        d[k][:200] = NAN
    d["out"], d["lse"] = binding.mla_prefill_bf16(d["q_nope"], d["q_rope"], d["k_nope"], d["k_rope"], d["v"], d["cu_q"],
                                                  d["cu_k"], SCALE)
    got = run(d)
    for x in got:
        assert bool(torch.isnan(x[:200]).all())
    check_rows(got, d, NAMES, list(range(200, 500)), "finite")


# lengths for which tiles of 256 queries would do, and others, with dS stored
@pytest.mark.parametrize("nq,nk,causal", [([1300], [1300], True), ([900, 1, 600], [1000, 3000, 2600], True),
                                          ([420, 410], [77, 1000], False), ([1, 900], [2, 900], False), ([385], [7000], True)],
                         ids=["1300", "mixed", "full", "one and 900", "385 of 7000"])
def test_gradients_of_stored_scores(cuda_device, nq, nk, causal):
    d = make(nq, nk, seed=25, causal=causal)
    ws = binding.alloc_workspace_prefill_backward(len(nq), sum(nq), sum(nk))
    got = run(d, causal, workspace=ws)
    check(got, d, causal, SCALE)
    for a, b in zip(run(d, causal, workspace=ws), got):
        assert torch.equal(a, b)
    assert binding.mla_get_status(ws) == 0


# more than 1024 tiles of scores, which find no room in the workspace: query tiles of 256 and of 128; and just 1024
LONG = [([520, 7], [33000, 70], True), ([520, 7], [33000, 70], False), ([300], [45000], True), ([140, 30], [60000, 18000], False),
        ([512], [32768], False)]


@pytest.mark.parametrize("nq,nk,causal", LONG, ids=["520 causal", "520 full", "300 causal", "140 and 30 full", "1024 tiles"])
def test_gradients_without_stored_scores(cuda_device, nq, nk, causal):
    d = make(nq, nk, seed=26, causal=causal)
    ws = binding.alloc_workspace_prefill_backward(len(nq), sum(nq), sum(nk))
    got = run(d, causal, workspace=ws)
    check(got, d, causal, SCALE)
    for a, b in zip(run(d, causal, workspace=ws), got):
        assert torch.equal(a, b)
    # the same workspace for short sequences, and back
    e = make([40, 200], [40, 250], seed=27)
    check(run(e, workspace=ws), e, True, SCALE)
    for a, b in zip(run(d, causal, workspace=ws), got):
        assert torch.equal(a, b)
    assert binding.mla_get_status(ws) == 0


@pytest.mark.parametrize("nq,nk", [(520, 33000), (300, 45000)], ids=["256", "128"])
@pytest.mark.parametrize("key", ["k_nope", "q_nope", "d_out"])
def test_masked_rows_without_stored_scores(cuda_device, nq, nk, key):
    d = make([nq], [nk], seed=28)
    row = 150
    if key == "k_nope":
        d[key][nk - nq + row] = NAN
    else:
        d[key][row] = NAN
    d["out"], d["lse"] = binding.mla_prefill_bf16(d["q_nope"], d["q_rope"], d["k_nope"], d["k_rope"], d["v"], d["cu_q"],
                                                  d["cu_k"], SCALE)
    got, exact = run(d), expected(d)
    check_rows(got, d, NAMES[:2], list(range(row)), key, exact)
    if key in ("q_nope", "d_out"):
        check_rows(got, d, NAMES[:2], list(range(row + 1, nq)), key, exact)
        check_rows(got, d, NAMES[2:], list(range(nk - nq + row + 1, nk)), key, exact)
