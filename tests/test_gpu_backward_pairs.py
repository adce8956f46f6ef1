"""The query pass on tiles of 256 rows (more than 1024 tiles of scores, long sequences on average): several sequences, causal
and full, against 64 bits.  Each case asserts that this form ran."""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from plain_backward import NAMES, check
from test_gpu_backward import SCALE, make, run
from test_gpu_backward_masked import check_rows, expected

pytestmark = pytest.mark.gpu

NAN = float("nan")


def workspace(nq, nk):
    return binding.alloc_workspace_prefill_backward(len(nq), sum(nq), sum(nk))


def assert_form(ws, stored, rows):
    """The plan behind the header: six counts, whether dq comes from stored tiles, and the rows of a query tile."""
    plan = ws[256:256 + 32].view(torch.int32).tolist()
    assert plan[6:8] == [stored, rows]


# tails of 32 and 80 keys; rows that see nothing and query tiles without steps; a sequence of one
CASES = [([520, 600], [20000, 18000], True), ([520, 600], [20000, 18000], False), ([2000, 700], [300, 30000], True),
         ([2000, 700], [300, 30000], False), ([600, 1, 800], [20000, 1, 20001], True), ([600, 1, 800], [20000, 1, 20001], False)]
IDS = [f"{a}x{b}{' causal' if c else ''}" for a, b, c in CASES]


@pytest.mark.parametrize("nq,nk,causal", CASES, ids=IDS)
def test_gradients_of_several_sequences(cuda_device, nq, nk, causal):
    d, ws = make(nq, nk, seed=len(nq) + nk[0], causal=causal), workspace(nq, nk)
    got = run(d, causal, workspace=ws)
    assert_form(ws, 0, 256)
    check(got, d, causal, SCALE)
    for a, b in zip(run(d, causal, workspace=ws), got):
        assert torch.equal(a, b)
    assert binding.mla_get_status(ws) == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bad", [0, 1], ids=["first", "second"])
def test_another_sequences_rows_do_not_matter(cuda_device, bad, causal):
    # the last tile of the first sequence's keys holds the second's first rows, and the last of its queries too
    nq, nk = [520, 600], [20000, 18000]
    d, ws = make(nq, nk, seed=31, causal=causal), workspace(nq, nk)
    want = run(d, causal, workspace=ws)
    assert_form(ws, 0, 256)
    spoilt = {k: x.clone() for k, x in d.items()}
    for k, n in (("q_nope", nq), ("q_rope", nq), ("d_out", nq), ("k_nope", nk), ("k_rope", nk), ("v", nk)):
        spoilt[k][slice(n[0] - 128, n[0]) if bad == 0 else slice(n[0], n[0] + 128)] = NAN
    spoilt["out"], spoilt["lse"] = binding.mla_prefill_bf16(
        *(spoilt[k] for k in ("q_nope", "q_rope", "k_nope", "k_rope", "v", "cu_q", "cu_k")), SCALE, causal=causal)
    got = run(spoilt, causal, workspace=ws)
    assert_form(ws, 0, 256)
    for a, b, n in zip(got, want, (nq, nq, nk, nk, nk)):
        other = slice(n[0], None) if bad == 0 else slice(0, n[0])
        assert torch.equal(a[other], b[other])


@pytest.mark.parametrize("key", ["k_nope", "k_rope", "q_nope", "d_out"])
def test_masked_rows_of_several_sequences(cuda_device, key):
    nq, nk, row = [520, 600], [20000, 18000], 300
    d, ws = make(nq, nk, seed=32), workspace(nq, nk)
    queries = key in ("q_nope", "d_out")
    for b in range(2):
        d[key][sum(nq[:b]) + row if queries else sum(nk[:b]) + nk[b] - nq[b] + row] = NAN
    d["out"], d["lse"] = binding.mla_prefill_bf16(d["q_nope"], d["q_rope"], d["k_nope"], d["k_rope"], d["v"], d["cu_q"],
                                                  d["cu_k"], SCALE)
    got, exact = run(d, workspace=ws), expected(d)
    assert_form(ws, 0, 256)
    for b in range(2):
        q0, k0 = sum(nq[:b]), sum(nk[:b])
        good = list(range(q0, q0 + row)) + (list(range(q0 + row + 1, q0 + nq[b])) if queries else [])
        check_rows(got, d, NAMES[:2], good, key, exact)
        if queries:
            check_rows(got, d, NAMES[2:], list(range(k0 + nk[b] - nq[b] + row + 1, k0 + nk[b])), key, exact)
