"""Backward pass at its limits: waits that run out, tensors at the end of the mapped memory, offsets past 4 GiB and more
sequences than a grid dimension has, and gradients against differences of the forward pass."""
import tempfile

import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import _build, binding
from plain_backward import NAMES, check
from test_gpu_backward import SCALE, make, run
from test_gpu_spans import Memory

pytestmark = pytest.mark.gpu

TIMEOUT = -6


@pytest.fixture(scope="module")
def stall_lib():
    d = tempfile.mkdtemp(prefix="mla_stall_backward_")
    return binding.load(_build.build(extra_flags=("-DMLA_WAIT_TIMEOUT_NS=2000000ull", "-DMLA_TEST_STALL_WAIT=1"),
                                     out_dir=d))


@pytest.mark.parametrize("nq,nk", [([300, 7], [300, 7]), ([300], [45000]), ([520], [33000])], ids=["stored", "128", "256"])
def test_a_wait_that_runs_out_ends_the_call_with_timeout_status(cuda_device, stall_lib, nq, nk):
    d = make(nq, nk, seed=31)
    ws = binding.alloc_workspace_prefill_backward(len(nq), sum(nq), sum(nk))
    want = run(d, workspace=ws)
    assert binding.mla_get_status(ws) == 0
    normal = binding.load()
    binding._lib = stall_lib
    try:
        run(d, workspace=ws)
        torch.cuda.synchronize()                      # the call returned: no hang
        assert binding.mla_get_status(ws) == TIMEOUT
    finally:
        binding._lib = normal
    for a, b in zip(run(d, workspace=ws), want):
        assert torch.equal(a, b)
    assert binding.mla_get_status(ws) == 0


@pytest.mark.parametrize("nq,nk", [([300, 7], [300, 70]), ([300], [45000])], ids=["stored", "not stored"])
def test_what_a_workspace_held_does_not_matter(cuda_device, nq, nk):
    d = make(nq, nk, seed=36)
    ws = binding.alloc_workspace_prefill_backward(len(nq), sum(nq), sum(nk))
    ws[256:] = 0
    want = run(d, workspace=ws)
    for byte in (0xFF, 0x7F):
        ws[256:] = byte
        for a, b in zip(run(d, workspace=ws), want):
            assert torch.equal(a, b)
    assert binding.mla_get_status(ws) == 0


def test_a_captured_call_with_a_workspace_of_its_own(cuda_device):
    d = make([150, 33], [150, 60], seed=37)
    want = run(d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(d)
    for _ in range(2):
        for x in got:
            x.fill_(7)
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 3, 200])
@pytest.mark.parametrize("name", ["d_out", "q_nope", "q_rope", "k_nope", "k_rope", "v", *NAMES])
def test_tensors_at_the_end_of_the_memory(cuda_device, n, name):
    memory = Memory(8 << 20)
    try:
        d = make([n], [n], seed=32)
        want = run(d)
        kw = {}
        if name in NAMES:
            kw[name] = memory.last(torch.zeros_like(want[NAMES.index(name)]))
        else:
            d[name] = memory.last(d[name].contiguous())
        for a, b in zip(run(d, **kw), want):
            assert torch.equal(a, b)
    finally:
        memory.free()


def test_many_sequences_and_offsets_past_4_gib(cuda_device):
    """65,536 sequences, the most of a call, of one or two tokens and one of 300; K, V and their gradients parts of wider rows."""
    rng = np.random.default_rng(33)
    n_k = rng.integers(1, 3, 65536)
    n_k[0] = 300
    n_q = np.minimum(n_k, rng.integers(0, 3, 65536))
    cu = [torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda") for n in (n_q, n_k)]
    tq, tk = int(n_q.sum()), int(n_k.sum())
    g = torch.Generator(device="cuda").manual_seed(33)
    q, kv, do, kr = (torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
                     for s in ((tq, 128, 192), (tk, 128, 256), (tq, 128, 128), (tk, 64)))
    assert kv.numel() > 1 << 31
    d = dict(q_nope=q[..., :128], q_rope=q[..., 128:], k_nope=kv[..., :128], k_rope=kr, v=kv[..., 128:], d_out=do,
             cu_q=cu[0], cu_k=cu[1])
    d["out"], d["lse"] = binding.mla_prefill_bf16(d["q_nope"], d["q_rope"], d["k_nope"], kr, d["v"], *cu, SCALE)
    dkv = torch.zeros_like(kv)
    got = run(d, dk_nope=dkv[..., :128], dv=dkv[..., 128:])
    for first in (0, 35000, 65529):                   # seven sequences each
        c = [x[first:first + 8].tolist() for x in cu]
        qs, ks = slice(c[0][0], c[0][-1]), slice(c[1][0], c[1][-1])
        part = {k: d[k][qs] for k in ("q_nope", "q_rope", "d_out", "out", "lse")}
        part |= {k: d[k][ks] for k in ("k_nope", "k_rope", "v")}
        part |= {"cu_q": [x - c[0][0] for x in c[0]], "cu_k": [x - c[1][0] for x in c[1]]}
        check([x[qs] for x in got[:2]] + [x[ks] for x in got[2:]], part, True, SCALE)
    # every sequence of a token has p = 1: dv = d_out
    one = np.flatnonzero((n_k == 1) & (n_q == 1))
    at_q, at_k = (torch.tensor(np.concatenate([[0], np.cumsum(n)])[one], device="cuda") for n in (n_q, n_k))
    for a, b in zip(at_q.split(8192), at_k.split(8192)):
        # (p = exp(s - lse) is 1 within 2^-11, which rounds to 1 in bf16; or to 1 - 2^-8)
        assert bool(((got[4][b].float() - do[a].float()).abs() <= 2.0 ** -7 * do[a].float().abs()).all())


def test_against_differences(cuda_device):
    """Directional derivatives of sum(d_out out) + sum(d_lse lse), the 64-bit forward taken from the formulas."""
    n_q, n_k = 24, 40
    d = make([n_q], [n_k], seed=34)
    d_lse = torch.randn((n_q, 128), generator=torch.Generator(device="cuda").manual_seed(34), device="cuda")
    got = dict(zip(NAMES, run(d, d_lse=d_lse)))
    see = torch.ones((n_q, n_k), dtype=torch.bool, device="cuda").tril(n_k - n_q)

    def value(x):
        q = torch.cat((x["q_nope"], x["q_rope"]), -1).transpose(0, 1)
        k = torch.cat((x["k_nope"].transpose(0, 1), x["k_rope"].expand(128, n_k, 64)), -1)
        s = (SCALE * q @ k.transpose(1, 2)).masked_fill(~see, -torch.inf)
        out = (torch.softmax(s, -1) @ x["v"].transpose(0, 1)).transpose(0, 1)
        return ((out * d["d_out"].double()).sum() + (torch.logsumexp(s, -1).T * d_lse.double()).sum()).item()

    at = {k: d[k].double() for k in ("q_nope", "q_rope", "k_nope", "k_rope", "v")}
    g = torch.Generator(device="cuda").manual_seed(35)
    for name, x in at.items():
        for _ in range(2):
            to = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
            eps = 1e-5
            slope = (value({**at, name: x + eps * to}) - value({**at, name: x - eps * to})) / (2 * eps)
            # every entry is off by its roundings, p's, ds's and its own, 3 * 2^-8 of terms that need not add up: along a
            # random direction their squares do, of a gradient whose terms are some times its size (40 terms: below 8)
            bound = 8 * 3 * 2.0 ** -8 * got["d" + name].double().norm().item()
            assert abs((got["d" + name].double() * to).sum().item() - slope) <= bound, name
