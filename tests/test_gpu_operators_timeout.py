"""The bounded waits of the kernels around the decode, made to run out without a
fault: in a copy of the library with a 2 ms limit and one wait in each kernel
that nothing completes, a call ends, its status is MLA_STATUS_TIMEOUT, and the
normal library gives the bits that it gave before in the same workspace."""
import tempfile

import pytest
import torch

from mla_latent_kv_05_gb300 import _build, binding
from test_gpu_operators_streams import Prefill, Tree

pytestmark = pytest.mark.gpu

TIMEOUT = -6


@pytest.fixture(scope="module")
def stall_lib():
    d = tempfile.mkdtemp(prefix="mla_stall_operators_")
    return binding.load(_build.build(extra_flags=("-DMLA_WAIT_TIMEOUT_NS=2000000ull", "-DMLA_TEST_STALL_WAIT=1"),
                                     out_dir=d))


def expand(p):
    return lambda: binding.mla_expand_kv(p.latent, *p.w, workspace=p.ews), p.ews


def prefill(p):
    k, v = binding.mla_expand_kv(p.latent, *p.w)
    return lambda: binding.mla_prefill_bf16(p.q, p.qr, k, p.kr, v, p.cu, p.cu, 192 ** -0.5, workspace=p.ws), p.ws


@pytest.mark.parametrize("kind", ["tree bf16", "tree fp8", "expand", "prefill"])
def test_a_wait_that_runs_out_ends_the_call_with_timeout_status(cuda_device, stall_lib, kind):
    if kind.startswith("tree"):
        t = Tree(kind[5:], 2)
        call, ws = t, t.ws
    else:
        call, ws = (expand if kind == "expand" else prefill)(Prefill(2))
    want = [x.clone() for x in call()]
    assert binding.mla_get_status(ws) == 0
    normal = binding.load()
    binding._lib = stall_lib
    try:
        call()
        torch.cuda.synchronize()                      # the call returned: no hang
        assert binding.mla_get_status(ws) == TIMEOUT
    finally:
        binding._lib = normal
    for a, b in zip(call(), want):
        assert torch.equal(a, b)
    assert binding.mla_get_status(ws) == 0
