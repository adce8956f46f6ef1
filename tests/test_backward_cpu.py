"""The backward pass of the expanded form without a GPU: the oracle's pins, and what the entry point refuses."""
import ctypes

import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import _build, binding
from oracle import expanded
from plain_backward import NAMES, backward

SCALE = 192 ** -0.5


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def head(n, m, seed, causal):
    r = np.random.default_rng(seed)
    q, k, v = r.standard_normal((n, 12)), r.standard_normal((m, 12)), r.standard_normal((m, 7))
    see = np.tril(np.ones((n, m), dtype=bool), m - n) if causal else np.ones((n, m), dtype=bool)
    return q, k, v, see, r.standard_normal((n, 7)), r.standard_normal(n)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,m", [(1, 1), (3, 5), (6, 4), (9, 9)])
def test_the_oracle_is_the_derivative_by_differences(n, m, causal):
    q, k, v, see, do, dl = head(n, m, n + m, causal)
    scale = 0.3

    def loss(q, k, v):
        out, lse, _ = expanded.attend(q, k, v, see, scale)
        return (out * do).sum() + (np.where(np.isfinite(lse), lse, 0.0) * dl).sum()

    out, lse, _ = expanded.attend(q, k, v, see, scale)
    got = expanded.attend_backward(q, k, v, see, scale, out, lse, do, dl)
    r = np.random.default_rng(1)
    for x, g in zip((0, 1, 2), got):
        for _ in range(4):
            step = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)]
            step[x] = r.standard_normal(step[x].shape)
            h = 1e-5
            by = (loss(q + h * step[0], k + h * step[1], v + h * step[2])
                  - loss(q - h * step[0], k - h * step[1], v - h * step[2])) / (2 * h)
            # central differences: h^2 of the third derivative, and 1e-16 / h of the loss
            assert abs(by - (g * step[x]).sum()) < 1e-8 * (1 + abs(by)) * 100


@pytest.mark.parametrize("causal", [True, False])
def test_the_oracle_is_autograds_gradient(causal):
    q, k, v, see, do, dl = head(11, 8, 3, causal)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    s = (0.3 * tq @ tk.T).masked_fill(~torch.tensor(see), -torch.inf)
    some = torch.tensor(see.any(1))
    lse = torch.logsumexp(s[some], -1)
    loss = ((torch.softmax(s[some], -1) @ tv) * torch.tensor(do)[some]).sum() + (lse * torch.tensor(dl)[some]).sum()
    loss.backward()
    out, l, _ = expanded.attend(q, k, v, see, 0.3)
    for got, want in zip(expanded.attend_backward(q, k, v, see, 0.3, out, l, do, dl), (tq, tk, tv)):
        assert np.abs(got - want.grad.numpy()).max() < 1e-12


def test_planted_mistakes_are_caught():
    q, k, v, see, do, dl = head(6, 6, 5, True)
    out, lse, _ = expanded.attend(q, k, v, see, 0.3)
    want = expanded.attend_backward(q, k, v, see, 0.3, out, lse, do, dl)

    def off(a, b):
        return max(np.abs(x - y).max() for x, y in zip(a, b))

    assert off(expanded.attend_backward(q, k, v, see, 0.3, 0 * out, lse, do, dl), want) > 1e-2      # no delta
    assert off(expanded.attend_backward(q, k, v, see, 0.3, out, lse, do, -dl), want) > 1e-2         # d_lse's sign
    assert off(expanded.attend_backward(q, k, v, np.ones_like(see), 0.3, out, lse, do, dl), want) > 1e-2
    assert off(expanded.attend_backward(q, k, v, see.T, 0.3, out, lse, do, dl), want) > 1e-2
    assert off(expanded.attend_backward(q, k, v, see, 0.3, out, lse / np.log(2), do, dl), want) > 1e-2


def problem(nq, nk, causal, seed):
    g = torch.Generator().manual_seed(seed)

    def r(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)

    d = dict(q_nope=r(sum(nq), 128, 128), q_rope=r(sum(nq), 128, 64), k_nope=r(sum(nk), 128, 128), k_rope=r(sum(nk), 64),
             v=r(sum(nk), 128, 128), d_out=r(sum(nq), 128, 128))
    d["cu_q"], d["cu_k"] = [0, *np.cumsum(nq).tolist()], [0, *np.cumsum(nk).tolist()]
    f = {k: x.double().numpy() for k, x in d.items() if isinstance(x, torch.Tensor)}
    out, lse, _ = expanded.prefill(f["q_nope"], f["q_rope"], f["k_nope"], f["k_rope"], f["v"], d["cu_q"], d["cu_k"], SCALE,
                                   causal, range(128))
    d["out"], d["lse"] = torch.from_numpy(out).to(torch.bfloat16), torch.from_numpy(lse).float()
    return d, torch.randn((sum(nq), 128), generator=g)


@pytest.mark.parametrize("causal", [True, False])
def test_the_plain_form_of_the_gpu_tests_is_the_oracle(causal):
    nq, nk = [3, 0, 5, 4], [4, 2, 3, 0]
    d, d_lse = problem(nq, nk, causal, 7)
    got, _ = backward(d, causal, SCALE, d_lse)
    want = dict(dq=np.zeros((12, 128, 192)), dk=np.zeros((9, 128, 192)), dv=np.zeros((9, 128, 128)))
    f = {k: x.double().numpy() for k, x in d.items() if isinstance(x, torch.Tensor)}
    for b in range(4):
        qs, ks = slice(d["cu_q"][b], d["cu_q"][b + 1]), slice(d["cu_k"][b], d["cu_k"][b + 1])
        see = np.ones((nq[b], nk[b]), dtype=bool)
        if causal:
            see = np.tril(see, nk[b] - nq[b])
        for h in range(128):
            q = np.concatenate([f["q_nope"][qs, h], f["q_rope"][qs, h]], -1)
            k = np.concatenate([f["k_nope"][ks, h], f["k_rope"][ks]], -1)
            want["dq"][qs, h], want["dk"][ks, h], want["dv"][ks, h] = expanded.attend_backward(
                q, k, f["v"][ks, h], see, SCALE, f["out"][qs, h], f["lse"][qs, h], f["d_out"][qs, h], d_lse.double().numpy()[qs, h])
    want = dict(dq_nope=want["dq"][..., :128], dq_rope=want["dq"][..., 128:], dk_nope=want["dk"][..., :128],
                dk_rope=want["dk"][..., 128:].sum(1), dv=want["dv"])
    for name in NAMES:
        assert np.abs(got[name].numpy() - want[name]).max() < 1e-11, name


def test_backward_entry_refuses_on_the_host(lib):
    fake, z = ctypes.c_void_p(0x1000), ctypes.c_void_p(0)
    odd = ctypes.c_void_p(0x1008)
    ok = (128 * 128, 128, 128 * 64, 64, 128 * 128, 128, 64, 128 * 128, 128, 128 * 128, 128, 128 * 128, 128, 128 * 64, 64,
          128 * 128, 128, 64, 128 * 128, 128)
    names = ["d_out", "d_lse", "q_nope", "q_rope", "k_nope", "k_rope", "v", "out", "lse", "strides", "cu_q", "cu_k", "batch",
             "num_q", "num_k", "num_heads", "causal", "scale", "dq_nope", "dq_rope", "dk_nope", "dk_rope", "dv", "ws", "n"]

    def call(strides=ok, **kw):
        a = {n: fake for n in names}
        a.update(d_lse=z, strides=(ctypes.c_size_t * 20)(*strides), batch=2, num_q=300, num_k=300, num_heads=128, causal=1,
                 scale=ctypes.c_float(0.1), n=1 << 40)
        a.update(kw)
        return lib.mla_prefill_backward_bf16(*[a[n] for n in names], z)

    for n in ("d_out", "q_nope", "q_rope", "k_nope", "k_rope", "v", "out", "dq_nope", "dq_rope", "dk_nope", "dk_rope", "dv"):
        assert call(**{n: z}) == -1 and call(**{n: odd}) == -1, n
    for n in ("lse", "cu_q", "cu_k", "ws", "strides"):
        assert call(**{n: z} if n != "strides" else dict(strides=(0,) * 20)) == -1, n
    assert call(d_lse=ctypes.c_void_p(0x1002)) == -1 and call(ws=ctypes.c_void_p(0x1080)) == -1
    for kw in (dict(batch=-1), dict(num_q=-1), dict(num_k=-1), dict(scale=ctypes.c_float(0.0)),
               dict(scale=ctypes.c_float(float("nan")))):
        assert call(**kw) == -1, kw
    assert call(num_heads=64) == -2 and call(batch=1 << 17) == -2 and call(num_q=1 << 25) == -2 and call(num_k=1 << 25) == -2
    for i in range(20):
        for bad in (0, 12, 1 << 40):
            s = list(ok)
            s[i] = bad
            assert call(strides=s) == -1, i
    n = ctypes.c_size_t(0)
    assert lib.mla_workspace_size_prefill_backward(2, 300, 300, ctypes.byref(n)) == 0
    assert call(n=n.value - 1) == -3
    assert call(batch=0) == 0 and call(num_q=0, num_k=0) == 0
    assert call() == -1                      # results in the place of inputs and of one another
    assert lib.mla_workspace_size_prefill_backward(2, 300, 300, None) == -1
    assert lib.mla_workspace_size_prefill_backward(-1, 300, 300, ctypes.byref(n)) == -1
    assert lib.mla_workspace_size_prefill_backward(1 << 17, 300, 300, ctypes.byref(n)) == -2
    assert binding.mla_workspace_size_prefill_backward(0, 0, 0) > 0
