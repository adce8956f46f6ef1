"""Calls on another stream than the current one that allocate their workspace
and outputs themselves: while they wait behind other work there, the current
stream allocates and fills memory of the same sizes, and each result is still
the bits of the call alone."""
import pytest
import torch

from test_gpu_operators_streams import Prefill, Rows, Tree
from mla_latent_kv_05_gb300 import binding

pytestmark = pytest.mark.gpu


def calls():
    t, f, p, r = Tree("bf16", 1), Tree("fp8", 2), Prefill(2), Rows(4)

    def tree(x):
        return lambda s: x.fn(*x.args, x.parents, x.scale, stream=s)

    def prefill(s):
        k, v = binding.mla_expand_kv(p.latent, *p.w, stream=s)
        return binding.mla_prefill_bf16(p.q, p.qr, k, p.kr, v, p.cu, p.cu, 192 ** -0.5, stream=s) + (k, v)

    def rows(s):
        binding.mla_cache_append_fp8(r.c, r.r, r.cache, *r.at, stream=s)
        return (binding.mla_cache_gather_fp8(r.cache, *r.at, 700, stream=s),)

    q4 = [x[:, :4].contiguous() for x in t.args[:2]]
    return [tree(t), tree(f), prefill, rows, lambda s: binding.mla_decode_bf16(*q4, *t.args[2:], t.scale, stream=s)]


def test_memory_of_a_call_on_a_side_stream_is_its_own(cuda_device):
    side = torch.cuda.Stream()
    for n, call in enumerate(calls()):
        want = [x.clone() for x in call(None)]
        sizes = sorted({x.numel() * x.element_size() for x in want} | {256, 1 << 20, 20 << 20, 40 << 20})
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)          # about 10 ms
            got = call(side)
            for _ in range(3):                         # what a freed block might be used for next
                for size in sizes:
                    torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
            torch.cuda.current_stream().wait_stream(side)
            bad = [int((x != y).sum()) for x, y in zip(got, want)]
            assert bad == [0] * len(want), (n, bad)
        torch.cuda.synchronize()
