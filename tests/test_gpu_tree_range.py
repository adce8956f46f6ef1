"""Tree decode straight from the codes of a quantised cache: what a page holds
behind the last token decides nothing."""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from mla_latent_kv_05_gb300 import inputs as gen
from test_gpu_tree import check, random_tree, reference, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "fp4", "fp8v41", "fp4v41"])
@pytest.mark.parametrize("fill", [0x00, 0x7F, 0xFF])
def test_rows_behind_the_end_do_not_change_the_pass(cuda_device, fmt, fill):
    lens = [70, 130, 64, 97]
    inp = gen.make_inputs(4, 6, lens, kv_dtype=fmt, seed=41)
    parents = random_tree(4, 6, 5)
    ref = reference(inp, parents)
    ws = binding.alloc_workspace_tree(4, 6)
    want = run(inp, parents, ws=ws)
    check(*want, *ref)
    live = torch.zeros(inp.kv_cache.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for tok in range(n):
            live[int(inp.block_table[b, tok // 64]), tok % 64] = True
    inp.kv_cache[~live] = fill
    # the same bits: the f16 pass answered both times, not the exact one
    got = run(inp, parents, ws=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
