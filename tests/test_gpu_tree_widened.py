"""Tree decode over quantised caches whose rows the workspace takes as bf16.

The widened rows are the codes times their power-of-two scale, which bf16
holds exactly at these magnitudes, so the bounds are those of the bf16 tree
decode (P and the result rounded once to bf16 each).
"""
import ctypes

import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from mla_latent_kv_05_gb300 import inputs as gen
from test_gpu_tree import check, random_tree, reference, run

pytestmark = pytest.mark.gpu

FORMATS = ["fp8", "fp4", "fp8v41", "fp4v41"]


def workspace(inp):
    return binding.alloc_workspace_tree(inp.batch, inp.sq, max_pages=inp.max_pages)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("t,lens", [(2, [2, 64, 65, 128, 191]), (7, [7, 70, 260]), (40, [100, 641]), (64, [64, 1500])])
def test_matches_float64(cuda_device, fmt, t, lens):
    inp = gen.make_inputs(len(lens), t, lens, kv_dtype=fmt, seed=5 * t + len(fmt))
    parents = random_tree(len(lens), t, t + 2)
    ws = workspace(inp)
    check(*run(inp, parents, ws=ws), *reference(inp, parents))
    assert binding.mla_get_status(ws) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_node_and_empty_sequences(cuda_device, fmt):
    inp = gen.make_inputs(4, 3, [3, 0, 200, 64], kv_dtype=fmt, seed=31)
    parents, n = random_tree(4, 3, 4), [3, 0, 1, 2]
    check(*run(inp, parents, n, ws=workspace(inp)), *reference(inp, parents, n))


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_behind_the_end_and_other_pages_may_hold_anything(cuda_device, fmt):
    lens = [70, 130, 64]
    inp = gen.make_inputs(3, 6, lens, kv_dtype=fmt, seed=32)
    parents = random_tree(3, 6, 5)
    ws = workspace(inp)
    want = run(inp, parents, ws=ws)
    live = torch.zeros(inp.kv_cache.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for tok in range(n):
            live[int(inp.block_table[b, tok // 64]), tok % 64] = True
    inp.kv_cache[~live] = 0xFF                         # NaN scales and codes
    ws[binding.mla_workspace_size_tree(3, 6):] = 0xFF
    got = run(inp, parents, ws=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_bad_page_is_recorded_and_reads_as_zeros(cuda_device):
    inp = gen.make_inputs(2, 5, [70, 200], kv_dtype="fp8", seed=33)
    parents = random_tree(2, 5, 6)
    ws = workspace(inp)
    want = run(inp, parents, ws=ws)
    inp.block_table[1, 1] = -3
    got = run(inp, parents, ws=ws)
    assert binding.mla_get_status(ws) == -5
    assert torch.equal(got[0][0], want[0][0])
    assert bool(torch.isfinite(got[0]).all())


def test_unseen_bad_rows_and_two_calls_in_one_workspace(cuda_device):
    inp = gen.make_inputs(2, 12, [12 + 90, 12 + 250], kv_dtype="fp8", seed=34)
    parents = random_tree(2, 12, 10)
    ws = workspace(inp)
    want, wl = run(inp, parents, ws=ws)
    tok = int(inp.seq_lens[1]) - 12 + 5
    inp.kv_cache[int(inp.block_table[1, tok // 64]), tok % 64] = 0x7F
    got, gl = run(inp, parents, ws=ws)
    for i in range(12):
        up, sees = i, False
        while up >= 0:
            sees |= up == 5
            up = int(parents[1, up])
        if sees:
            assert torch.isnan(got[1, i]).all()
        else:
            assert torch.equal(got[1, i], want[1, i]) and torch.equal(gl[1, i], wl[1, i]), i
    assert torch.equal(got[0], want[0])


def test_a_workspace_one_byte_short_reads_the_codes_directly(cuda_device):
    inp = gen.make_inputs(2, 4, [40, 300], kv_dtype="fp4", seed=35)
    parents = random_tree(2, 4, 7)
    ref = reference(inp, parents)
    full = workspace(inp)
    check(*run(inp, parents, ws=full), *ref)
    check(*run(inp, parents, ws=full[:-1]), *ref)


def test_captured_graph_over_a_cache_that_grows(cuda_device):
    inp = gen.make_inputs(2, 4, [60, 300], kv_dtype="fp8", seed=36)
    parents = random_tree(2, 4, 8).cuda()
    ws = workspace(inp)
    q, qr, kv, bt, sl = (x.cuda() for x in (inp.q_absorbed, inp.q_rope, inp.kv_cache, inp.block_table, inp.seq_lens))
    out = torch.empty((2, 4, 128, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 4, 128), device="cuda")

    def call():
        binding.mla_decode_tree_fp8(q, qr, kv, bt, sl, parents, inp.scale, out=out, lse=lse, workspace=ws)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([9, 100], [60, 300], [4, 65]):
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        inp.seq_lens = torch.tensor(lens, dtype=torch.int32)
        check(out, lse, *reference(inp, parents.cpu()))
    assert binding.mla_get_status(ws) == 0


def test_size_of_the_workspace(cuda_device):
    small = binding.mla_workspace_size_tree(3, 5)
    assert binding.mla_workspace_size_tree_widened(3, 5, 7) == small + 3 * 7 * 64 * 576 * 2
    n = ctypes.c_size_t(0)
    lib = binding.load()
    assert lib.mla_workspace_size_tree_widened(3, 5, 128, 64, 0, ctypes.byref(n)) == -1
    assert lib.mla_workspace_size_tree_widened(3, 65, 128, 64, 7, ctypes.byref(n)) == -2
