"""Gradients of the expanded-form attention on the GPU against the formulas in 64 bits (bounds: plain_backward.py)."""
import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from plain_backward import NAMES, check

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def make(nq, nk, seed, causal=True, behind=0, amp=1.0):
    """Inputs on the GPU, out and lse from the forward entry; `behind`: rows of no sequence, NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(n, *shape):
        x = torch.randn((n + behind, *shape), generator=g, device="cuda").to(torch.bfloat16)
        x[n:] = float("nan")
        return x

    tq, tk = sum(nq), sum(nk)
    q, rows = r(tq, 128, 192) * amp, r(tk, 576)
    d = dict(q_nope=q[..., :128], q_rope=q[..., 128:], k_nope=r(tk, 128, 128), k_rope=rows[:, 512:], v=r(tk, 128, 128),
             d_out=r(tq, 128, 128))
    d["cu_q"] = torch.tensor(np.concatenate([[0], np.cumsum(nq)]), dtype=torch.int32, device="cuda")
    d["cu_k"] = torch.tensor(np.concatenate([[0], np.cumsum(nk)]), dtype=torch.int32, device="cuda")
    out = torch.full((tq + behind, 128, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tq + behind, 128), float("nan"), device="cuda")
    d["out"], d["lse"] = binding.mla_prefill_bf16(d["q_nope"], d["q_rope"], d["k_nope"], d["k_rope"], d["v"], d["cu_q"],
                                                  d["cu_k"], SCALE, causal=causal, out=out, lse=lse)
    return d


def run(d, causal=True, **kw):
    return binding.mla_prefill_backward_bf16(d["d_out"], d["q_nope"], d["q_rope"], d["k_nope"], d["k_rope"], d["v"], d["out"],
                                             d["lse"], d["cu_q"], d["cu_k"], SCALE, causal=causal, **kw)


CASES = [([1], [1]), ([2], [1]), ([1], [2]), ([33, 7, 1, 20, 5], [33, 7, 1, 20, 5]), ([128], [128]), ([127], [129]),
         ([129, 128, 127], [129, 128, 127]), ([256, 1], [256, 300]), ([300], [700]), ([5, 0, 64], [900, 130, 0]),
         ([513], [513]), ([700, 30], [40, 1000])]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", CASES, ids=[f"{a}x{b}" for a, b in CASES])
def test_gradients(cuda_device, nq, nk, causal):
    d = make(nq, nk, seed=sum(nq) + 31 * sum(nk), causal=causal)
    ws = binding.alloc_workspace_prefill_backward(len(nq), sum(nq), sum(nk))
    got = run(d, causal, workspace=ws)
    check(got, d, causal, SCALE)
    assert binding.mla_get_status(ws) == 0
    # the same bits again, in a workspace that was used
    for a, b in zip(run(d, causal, workspace=ws), got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", [([1000], [1000]), ([1111, 400, 64, 2, 900], [1111, 1500, 64, 3, 900])], ids=["1000", "ragged"])
def test_gradients_of_longer_sequences(cuda_device, nq, nk, causal):
    d = make(nq, nk, seed=9, causal=causal)
    check(run(d, causal), d, causal, SCALE)


@pytest.mark.parametrize("causal", [True, False])
def test_gradient_of_the_lse(cuda_device, causal):
    d = make([150, 40], [150, 200], seed=4, causal=causal)
    d_lse = torch.randn((190, 128), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    got = run(d, causal, d_lse=d_lse)
    check(got, d, causal, SCALE, d_lse)
    zero = run(d, causal, d_lse=torch.zeros_like(d_lse))
    for a, b in zip(zero, run(d, causal)):
        assert torch.equal(a, b)


def test_sharp_scores(cuda_device):
    # scores of up to about 60: p from 1 down to nothing
    d = make([300, 40], [300, 500], seed=5, amp=8.0)
    # (a score's fp32 sum is eight times as large here, and so is its error: q is scaled by a power of two, so the bound's
    # 2^-10 for the exponential becomes 2^-8 at most; the bf16 roundings stay, so the bound is doubled)
    from plain_backward import backward
    want, bound = backward(d, True, SCALE)
    for name, x in zip(NAMES, run(d)):
        assert bool(((x.double() - want[name]).abs() <= 2 * bound[name]).all()), name


def test_rows_of_no_sequence_are_left_alone(cuda_device):
    d = make([70, 200], [150, 200], seed=6, behind=9)
    shapes = ((279, 128, 128), (279, 128, 64), (359, 128, 128), (359, 64), (359, 128, 128))
    grads = [torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for s in shapes]
    got = run(d, **dict(zip(NAMES, grads)))
    for a, b in zip(got, grads):
        assert a is b and bool((a[-9:] == 7).all())
    check(got, d, True, SCALE)


def test_views_in_and_out(cuda_device):
    d = make([140, 3], [140, 260], seed=7)
    want = run(d)
    dq = torch.zeros((143, 128, 192), dtype=torch.bfloat16, device="cuda")
    dkv = torch.zeros((400, 128, 256), dtype=torch.bfloat16, device="cuda")
    dc = torch.zeros((400, 576), dtype=torch.bfloat16, device="cuda")
    e = {k: x.contiguous() if x.dim() > 1 else x for k, x in d.items()}
    e["d_out"] = d["d_out"].transpose(0, 1).contiguous().transpose(0, 1)
    got = run(e, dq_nope=dq[..., :128], dq_rope=dq[..., 128:], dk_nope=dkv[..., :128], dv=dkv[..., 128:], dk_rope=dc[:, 512:])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(dq[..., 128:], want[1]) and torch.equal(dc[:, 512:], want[3]) and not dc[:, :512].any()


def test_no_keys_and_no_queries(cuda_device):
    d = make([40], [0], seed=8)
    got = run(d)
    assert not got[0].any() and not got[1].any() and got[2].shape == (0, 128, 128)
    e = make([0, 0], [30, 100], seed=8)
    got = run(e)
    assert got[0].shape == (0, 128, 128) and not any(bool(x.any()) for x in got[2:])
    n = make([], [], seed=1)
    assert [x.shape[0] for x in run(n)] == [0] * 5


@pytest.mark.parametrize("where", ["cu_q", "cu_k"])
def test_a_sequence_with_bad_bounds_is_skipped(cuda_device, where):
    d = make([100, 60, 30], [100, 60, 30], seed=9)
    ws = binding.alloc_workspace_prefill_backward(3, 190, 190)
    good = run(d, workspace=ws)
    bad = dict(d)
    bad[where] = d[where].clone()
    bad[where][3] = 500
    grads = [torch.full_like(x, 7.0) for x in good]
    got = run(bad, workspace=ws, **dict(zip(NAMES, grads)))
    assert binding.mla_get_status(ws) == -7
    for a, b in zip(got, good):
        assert torch.equal(a[:160], b[:160]) and bool((a[160:] == 7).all())
    assert binding.mla_get_status(ws) == 0
    for a, b in zip(run(d, workspace=ws), good):
        assert torch.equal(a, b)


def test_refusals(cuda_device):
    d = make([10], [12], seed=10)
    for k, x, err in (("d_out", d["d_out"].float(), TypeError), ("d_out", d["d_out"][:9], ValueError),
                      ("out", d["out"][:9], ValueError), ("out", d["out"].transpose(0, 1), ValueError),
                      ("lse", d["lse"].half(), TypeError), ("lse", d["lse"][:9], ValueError),
                      ("v", d["v"][:11], ValueError), ("q_rope", d["q_rope"].cpu(), ValueError),
                      ("cu_k", d["cu_k"][:1], ValueError), ("cu_q", d["cu_q"].long(), TypeError),
                      ("d_out", d["d_out"][:, :1].expand(10, 128, 128), ValueError)):
        with pytest.raises(err):
            run({**d, k: x})
    with pytest.raises(ValueError):
        run(d, dv=torch.zeros((11, 128, 128), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        run(d, d_lse=torch.zeros((10, 128), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(binding.MLAError):
        run(d, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(binding.MLAError):
        binding.mla_prefill_backward_bf16(d["d_out"], d["q_nope"], d["q_rope"], d["k_nope"], d["k_rope"], d["v"], d["out"],
                                          d["lse"], d["cu_q"], d["cu_k"], 0.0)


def test_on_another_stream_and_in_a_captured_graph(cuda_device):
    d = make([200, 30], [200, 90], seed=11)
    want = run(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(d, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    ws = binding.alloc_workspace_prefill_backward(2, 230, 290)
    grads = [torch.zeros_like(x) for x in want]
    run(d, workspace=ws)
    graphs = []
    for _ in range(2):                                # two graphs that share a workspace, replayed in order
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(d, workspace=ws, **dict(zip(NAMES, grads)))
        graphs.append(graph)
    for graph in (*graphs, *graphs):
        for x in grads:
            x.zero_()
        graph.replay()
        for a, b in zip(grads, want):
            assert torch.equal(a, b)


def test_two_calls_at_once(cuda_device):
    ds = [make([300], [300], seed=12), make([257, 40], [300, 40], seed=13)]
    want = [run(d) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(d, stream=s) for d, s in zip(ds, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for a, b in zip(g, w):
                assert torch.equal(a, b)


def test_rotation_attention_and_their_gradients_in_a_row(cuda_device):
    """One training step of the expanded form: rotate, attend, and back through both."""
    from oracle import expanded, rope
    g = torch.Generator().manual_seed(14)
    n = 40
    q, k, v = (torch.randn(s, generator=g).to(torch.bfloat16) for s in ((n, 128, 192), (n, 128, 128), (n, 128, 128)))
    kr, do = torch.randn((n, 64), generator=g).to(torch.bfloat16), torch.randn((n, 128, 128), generator=g).to(torch.bfloat16)
    f = rope.frequencies()
    t = binding.mla_rope_init(f)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    qg, kg, vg, krg, dog = (x.cuda() for x in (q, k, v, kr, do))
    q_rot, k_rot = binding.mla_rope_bf16(qg[..., 128:], pos, t), binding.mla_rope_bf16(krg, pos, t)
    out, lse = binding.mla_prefill_bf16(qg[..., :128], q_rot, kg, k_rot, vg, cu, cu, SCALE)
    dqn, dqr, dkn, dkr, dv = binding.mla_prefill_backward_bf16(dog, qg[..., :128], q_rot, kg, k_rot, vg, out, lse, cu, cu, SCALE)
    dq_rope, dk_rope = (binding.mla_rope_bf16(x, pos, t, inverse=True) for x in (dqr, dkr))
    # the whole of it in 64 bits, unrounded between the steps, by autograd on angles as products
    a = {}
    for name, x in (("q", q), ("k", k), ("v", v), ("kr", kr)):
        a[name] = x.double().requires_grad_()
    angle = torch.outer(torch.arange(n, dtype=torch.float64), torch.tensor(f, dtype=torch.float64))

    def rot(x):
        c, s = torch.cos(angle), torch.sin(angle)
        while c.dim() < x.dim():
            c, s = c.unsqueeze(1), s.unsqueeze(1)
        return torch.stack((x[..., 0::2] * c - x[..., 1::2] * s, x[..., 0::2] * s + x[..., 1::2] * c), -1).flatten(-2)

    qf = torch.cat((a["q"][..., :128], rot(a["q"][..., 128:])), -1).transpose(0, 1)
    kf = torch.cat((a["k"].transpose(0, 1), rot(a["kr"]).expand(128, n, 64)), -1)
    s = (SCALE * qf @ kf.transpose(1, 2)).masked_fill(~torch.ones(n, n).tril().bool(), -torch.inf)
    ((torch.softmax(s, -1) @ a["v"].transpose(0, 1)).transpose(0, 1) * do.double()).sum().backward()
    # every step's roundings, each 2^-8 of a value of the result's size: rotated inputs, out, p, ds, two results
    for got, want in ((dqn, a["q"].grad[..., :128]), (dq_rope, a["q"].grad[..., 128:]), (dkn, a["k"].grad),
                      (dk_rope, a["kr"].grad), (dv, a["v"].grad)):
        off = (got.double().cpu() - want).norm() / want.norm()
        assert off < 6 * 2.0 ** -8, off
