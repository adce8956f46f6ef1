"""The sequence of each packed row, where few of many sequences hold any: rows
whose sequences lie more than 32 apart, on both sides of a long call's rule."""
import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,density,most,seed", [(1, 1.0, 5, 0), (31, 1.0, 3, 1), (32, 0.5, 3, 2), (33, 0.3, 40, 3),
                                                     (200, 0.02, 3, 4), (1500, 0.02, 2, 5), (1500, 1.0, 9, 6),
                                                     (4000, 0.004, 700, 7), (700, 1.0, 40, 8)])
def test_rows_land_at_their_sequences_tokens(cuda_device, batch, density, most, seed):
    rng = np.random.default_rng(seed)
    n = np.where(rng.random(batch) < density, rng.integers(1, most + 1, batch), 0)
    n[rng.integers(batch)] += 1                              # at least one row
    cu = np.concatenate([[0], np.cumsum(n)])
    rows = int(cu[-1])
    lens = n + rng.integers(0, 70, batch)
    pages = max(1, int(np.ceil(lens.max() / 64)))
    table = rng.permutation(batch * pages).reshape(batch, pages)
    g = torch.Generator().manual_seed(seed)
    c = torch.randn((rows + 5, 512), generator=g).to(torch.bfloat16).cuda()
    r = torch.randn((rows + 5, 64), generator=g).to(torch.bfloat16).cuda()
    cache = torch.zeros((batch * pages, 64, 576), dtype=torch.bfloat16, device="cuda")

    def ints(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = cache, ints(table), ints(lens), ints(cu)
    binding.mla_cache_append_bf16(c, r, *args, workspace=ws)
    b = np.repeat(np.arange(batch), n)
    pos = lens[b] - cu[b + 1] + np.arange(rows)
    at = torch.tensor(table[b, pos // 64] * 64 + pos % 64, device="cuda")
    want = torch.zeros_like(cache).view(-1, 576)
    want[at] = torch.cat([c, r], 1)[:rows]
    assert torch.equal(cache.view(-1, 576), want)
    out = torch.full((rows + 5, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.mla_cache_gather_bf16(*args, rows + 5, out=out, workspace=ws)
    assert torch.equal(out[:rows], torch.cat([c, r], 1)[:rows]) and bool((out[rows:] == 7).all())
    assert binding.mla_get_status(ws) == 0
