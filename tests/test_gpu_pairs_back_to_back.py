"""The kernels that run on pairs of CTAs, in short calls one behind the other and
on two streams, so that a pair's successors start in its shared memory the
moment it has left: every call gives the bits of the first one."""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from mla_latent_kv_05_gb300 import inputs as gen
from test_gpu_tree import random_tree

pytestmark = pytest.mark.gpu


def expand_call(n, seed):
    g = torch.Generator().manual_seed(seed)
    rows, uk, uv = ((torch.randn(s, generator=g) * f).to(torch.bfloat16).cuda()
                    for s, f in (((n, 512), 1.0), ((128, 128, 512), 512 ** -0.5), ((128, 128, 512), 512 ** -0.5)))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return lambda: binding.mla_expand_kv(rows, uk, uv, workspace=ws), ws


def tree_call(fmt, t, lens, seed):
    inp = gen.make_inputs(len(lens), t, lens, kv_dtype=fmt, seed=seed)
    args = [x.cuda() for x in (inp.q_absorbed, inp.q_rope, inp.kv_cache, inp.block_table, inp.seq_lens,
                               random_tree(len(lens), t, seed))]
    ws = binding.alloc_workspace_tree(len(lens), t, max_pages=0 if fmt == "bf16" else inp.max_pages)
    fn = getattr(binding, "mla_decode_tree_" + fmt)
    return lambda: fn(*args, inp.scale, workspace=ws), ws


def test_short_calls_in_a_row_and_on_two_streams(cuda_device):
    sets = [[expand_call(1, 1), tree_call("bf16", 3, [9, 70], 2), expand_call(130, 3), tree_call("fp8", 5, [300], 4)],
            [tree_call("bf16", 1, [64], 5), expand_call(257, 6), tree_call("fp4", 2, [5, 400, 64], 7)]]
    want = [[[x.clone() for x in call()] for call, _ in s] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    bad = []
    for s, stream in zip(sets, streams):
        with torch.cuda.stream(stream):
            bad.append(torch.zeros((), dtype=torch.int64, device="cuda"))
    for _ in range(60):
        for s, w, stream, n in zip(sets, want, streams, bad):
            with torch.cuda.stream(stream):
                got = [call() for call, _ in s]
                for a, b in zip(got, w):
                    for x, y in zip(a, b):
                        n += (x != y).sum()
    torch.cuda.synchronize()
    assert [int(n) for n in bad] == [0, 0]
    for s in sets:
        for _, ws in s:
            assert binding.mla_get_status(ws) == 0
