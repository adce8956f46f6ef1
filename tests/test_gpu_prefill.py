"""Expanded-form attention on the GPU against the float64 oracle.

Bound per output element: P is rounded to bf16 (2^-8 of sum p|v|), the result
once more (2^-8 of |out|), and the fp32 scores (192 products, 192 * 2^-23 of
scale * sum|q||k|, about 2e-4 on these inputs, taken twice: numerator and
denominator) are worth 2^-10 of sum p|v|.  lse: 1e-3 absolute, from the same
score error.
"""
import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from oracle import expanded

pytestmark = pytest.mark.gpu

SCALE = 1.0 / 192 ** 0.5
HEADS = [0, 1, 63, 127]


def make(nq, nk, seed, packed=True, amp=1.0):
    g = torch.Generator().manual_seed(seed)

    def r(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)

    tq, tk = sum(nq), sum(nk)
    q, rows = r(tq, 128, 192) * amp, r(tk, 576)
    d = dict(q_nope=q[..., :128], q_rope=q[..., 128:], k_nope=r(tk, 128, 128), k_rope=rows[:, 512:], v=r(tk, 128, 128))
    if not packed:
        d = {k: v.contiguous() for k, v in d.items()}
    d["cu_q"] = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32)
    d["cu_k"] = torch.tensor(np.concatenate([[0], np.cumsum(nk)]), dtype=torch.int32)
    return d


def cuda(d, packed=True):
    out = {}
    for k, v in d.items():
        if packed and v.dim() >= 2 and not v.is_contiguous():
            base = torch.empty_strided((v.shape[0],) + tuple(v.shape[1:]), v.stride(), dtype=v.dtype, device="cuda")
            base.copy_(v)
            out[k] = base
        else:
            out[k] = v.cuda()
    return out


def run(d, causal=True, **kw):
    return binding.mla_prefill_bf16(d["q_nope"], d["q_rope"], d["k_nope"], d["k_rope"], d["v"], d["cu_q"], d["cu_k"],
                                    SCALE, causal=causal, **kw)


def check(out, lse, d, causal, heads=HEADS):
    f = {k: v.double().numpy() for k, v in d.items()}
    ref, rl, mag = expanded.prefill(f["q_nope"], f["q_rope"], f["k_nope"], f["k_rope"], f["v"], d["cu_q"], d["cu_k"],
                                    SCALE, causal, heads)
    got = out.double().cpu().numpy()[:, heads]
    gl = lse.double().cpu().numpy()[:, heads]
    own = ~np.isnan(rl)
    np.testing.assert_array_equal(np.isneginf(gl[own]), np.isneginf(rl[own]))
    fin = own & np.isfinite(rl)
    assert np.abs(gl[fin] - rl[fin]).max(initial=0) <= 1e-3
    bound = (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -8 * np.abs(ref)
    err = np.abs(got - ref)
    assert (err[own] <= bound[own] + 1e-30).all(), np.nanmax(err - bound)


def status_run(d, causal=True):
    ws = binding.alloc_workspace_prefill(d["cu_q"].numel() - 1, d["q_nope"].shape[0])
    out, lse = run(d, causal, workspace=ws)
    assert binding.mla_get_status(ws) == 0
    return out, lse


CASES = [
    ([1], [1]),
    ([1, 1, 1], [1, 130, 64]),
    ([3, 33, 17, 1, 5], [3, 33, 17, 1, 5]),
    ([127], [127]), ([128], [128]), ([129], [129]), ([255], [255]), ([256], [256]), ([257], [257]),
    ([300, 20, 128], [300, 150, 700]),     # prompts, and chunks over a cached context
    ([140, 0, 3], [20, 5, 0]),             # more queries than keys, no query, no key
    ([400], [130]),                        # a whole tile of queries that see nothing
    ([600], [900]),
]


@pytest.mark.parametrize("nq,nk", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_matches_the_oracle(cuda_device, nq, nk, causal):
    d = make(nq, nk, sum(nq) + 7 * sum(nk))
    out, lse = status_run(cuda(d), causal)
    check(out, lse, d, causal)


def test_contiguous_and_head_major_inputs_agree(cuda_device):
    d = make([200, 31], [250, 31], 3)
    a, la = run(cuda(d))
    b, lb = run({k: v.cuda().contiguous() for k, v in d.items()})
    assert torch.equal(a, b) and torch.equal(la, lb)
    hm = {k: v.cuda().contiguous() for k, v in d.items()}
    for k in ("q_nope", "q_rope", "k_nope", "v"):
        hm[k] = hm[k].transpose(0, 1).contiguous().transpose(0, 1)       # [H, n, d] in memory
    c, lc = run(hm)
    assert torch.equal(a, c) and torch.equal(la, lc)


def test_large_scores_move_the_reference_often(cuda_device):
    # keys whose scores rise along the sequence, far beyond the lazy bound
    d = make([70, 300], [500, 300], 4, amp=4.0)
    ramp = torch.linspace(0.1, 12.0, 800)[:, None, None]
    d["k_nope"] = (d["k_nope"].float() * ramp).to(torch.bfloat16)
    out, lse = status_run(cuda(d))
    f = {k: v.double().numpy() for k, v in d.items()}
    ref, rl, mag = expanded.prefill(f["q_nope"], f["q_rope"], f["k_nope"], f["k_rope"], f["v"], d["cu_q"], d["cu_k"],
                                    SCALE, True, HEADS)
    # |score| <= scale * sum|q||k| ~ 0.072 * 192 * 4 * 12 * 0.64 ~ 430 here: 192 * 2^-23 of it is 1e-2 per score
    err = np.abs(out.double().cpu().numpy()[:, HEADS] - ref)
    assert (err <= (2.0 ** -8 + 2e-2) * mag + 2.0 ** -8 * np.abs(ref)).all()
    assert np.abs(lse.double().cpu().numpy()[:, HEADS] - rl).max() <= 1e-2


def test_other_sequences_and_masked_keys_do_not_reach_a_query(cuda_device):
    d = make([100, 60, 90], [100, 60, 90], 5)
    want, wl = run(cuda(d))
    e = {k: v.clone() for k, v in d.items()}
    for k in ("k_nope", "v", "k_rope"):
        e[k][100:160] = float("nan")                       # the middle sequence is all NaN
    e["k_nope"][99] = float("inf")                         # the last key of the first: its last query alone sees it
    got, gl = run(cuda(e))
    keep = list(range(0, 99)) + list(range(160, 250))
    assert torch.equal(got[keep], want[keep]) and torch.equal(gl[keep], wl[keep])
    assert torch.isnan(got[100:160]).all()


def test_rows_behind_the_last_sequence_stay(cuda_device):
    d = make([40, 30], [40, 30], 6)
    d["cu_q"] = torch.tensor([0, 40], dtype=torch.int32)
    d["cu_k"] = torch.tensor([0, 40], dtype=torch.int32)
    c = cuda(d)
    out = torch.full((70, 128, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((70, 128), 3.0, device="cuda")
    run(c, out=out, lse=lse)
    assert bool((out[40:] == 3).all()) and bool((lse[40:] == 3).all())
    check(out[:40], lse[:40], {k: (v[:40] if v.dim() > 1 else v) for k, v in d.items()}, True)


def test_bad_bounds_are_recorded_and_skipped(cuda_device):
    d = make([40, 30, 20], [40, 30, 20], 7)
    c = cuda(d)
    good, _ = run(c)
    for name, bad in (("cu_q", [0, 40, 95, 90]), ("cu_k", [0, -1, 70, 90]), ("cu_q", [0, 200, 70, 90])):
        e = dict(c)
        e[name] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        ws = binding.alloc_workspace_prefill(3, 90)
        out = torch.full((90, 128, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        run(e, out=out, workspace=ws)
        assert binding.mla_get_status(ws) == -7
        if name == "cu_q" and bad[1] == 40:
            assert torch.equal(out[:40], good[:40]) and bool((out[40:] == 3).all())


def test_many_short_sequences(cuda_device):
    nq = [1 + i % 4 for i in range(230)]
    nk = [n + i % 37 for i, n in enumerate(nq)]
    d = make(nq, nk, 8)
    out, lse = status_run(cuda(d))
    check(out, lse, d, True, heads=[5, 100])


@pytest.mark.parametrize("nq,nk", [([300] * 12 + [700, 5], [0] * 12 + [10, 9]), ([900, 260, 900], [100, 600, 3])])
def test_runs_of_tiles_without_keys(cuda_device, nq, nk):
    # many tiles whose queries see nothing, between tiles that have work
    d = make(nq, nk, 13)
    out, lse = status_run(cuda(d))
    check(out, lse, d, True, heads=[0, 77])


def test_captured_graph_two_streams_and_repeatability(cuda_device):
    d = make([300, 45], [420, 45], 9)
    c = cuda(d)
    want, wl = run(c)
    ws = binding.alloc_workspace_prefill(2, 345)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    run(c, out=out, lse=lse, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(c, out=out, lse=lse, workspace=ws)
    e = make([300, 45], [420, 45], 10)
    ec = cuda(e)
    want2, wl2 = run(ec)
    for k in ("q_nope", "q_rope", "k_nope", "k_rope", "v"):
        c[k].copy_(ec[k])
    g.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws2 = binding.alloc_workspace_prefill(2, 345)
    o2, l2 = run(c, workspace=ws2, stream=s)               # beside the graph, on a workspace of its own
    torch.cuda.synchronize()
    assert binding.mla_get_status(ws) == 0 and binding.mla_get_status(ws2) == 0
    assert torch.equal(out, want2) and torch.equal(lse, wl2)
    assert torch.equal(o2, want2) and torch.equal(l2, wl2)


def test_long_context_matches_float64_on_the_gpu(cuda_device):
    # 5 queries over 9000 keys, and a 1500-token prompt, all heads
    d = make([5, 1500], [9000, 1500], 11)
    c = cuda(d)
    out, lse = status_run(c)
    q0 = k0 = 0
    for nq, nk in ((5, 9000), (1500, 1500)):
        see = torch.ones((nq, nk), dtype=torch.bool, device="cuda").tril(nk - nq)
        for h in range(0, 128, 9):
            q = torch.cat([c["q_nope"][q0:q0 + nq, h], c["q_rope"][q0:q0 + nq, h]], -1).double()
            k = torch.cat([c["k_nope"][k0:k0 + nk, h], c["k_rope"][k0:k0 + nk]], -1).double()
            s = (q @ k.T * SCALE).masked_fill(~see, -torch.inf)
            p = torch.softmax(s, -1)
            v = c["v"][k0:k0 + nk, h].double()
            ref, mag = p @ v, p @ v.abs()
            err = (out[q0:q0 + nq, h].double() - ref).abs()
            assert bool((err <= (2.0 ** -8 + 2.0 ** -10) * mag + 2.0 ** -8 * ref.abs()).all())
            assert float((lse[q0:q0 + nq, h].double() - torch.logsumexp(s, -1)).abs().max()) <= 1e-3
        q0, k0 = q0 + nq, k0 + nk
