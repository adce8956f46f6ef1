"""Tree decode straight from the codes where the f16 pass cannot answer: a query
or a cached value beyond f16 makes it hold infinities, whose products with zeros
are NaN, so that only the pass with bf16 operands gives the numbers checked here.

Bound per element: P is rounded to bf16 (2^-8 of sum p|v|), the result once more
(2^-8 of |out|); the fp32 scores (576 products of unit normal values: an error
of 576 * 2^-24 * scale * sum|q||k| < 1e-3, twice) are worth 2^-9 of sum p|v|.
lse: 1e-3.
"""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from test_gpu_tree import random_tree
from oracle import expanded

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
FORMATS = ["fp8", "fp4", "fp8_v41", "fp4_v41"]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(fmt, lens, t, seed, prepare):
    g = torch.Generator().manual_seed(seed)
    total, pages = sum(lens), -(-max(lens) // 64)
    c, kr = torch.randn((total, 512), generator=g), torch.randn((total, 64), generator=g)
    q, qr = torch.randn((len(lens), t, 128, 512), generator=g), torch.randn((len(lens), t, 128, 64), generator=g)
    prepare(c, q)
    c, kr, q, qr = (x.to(torch.bfloat16).cuda() for x in (c, kr, q, qr))
    table = torch.randperm(len(lens) * pages, generator=g).to(torch.int32).view(len(lens), pages).cuda()
    cache = torch.zeros((len(lens) * pages, 64, binding._ROW_WIDTH[fmt]), dtype=torch.uint8, device="cuda")
    cu = ints([0] + [sum(lens[:b + 1]) for b in range(len(lens))])
    getattr(binding, "mla_cache_append_" + fmt)(c, kr, cache, table, ints(lens), cu)
    rows = getattr(binding, "mla_cache_gather_" + fmt)(cache, table, ints(lens), cu, total)
    parents = random_tree(len(lens), t, seed)
    ws = binding.alloc_workspace_tree(len(lens), t)           # no room for widened rows
    out, lse = getattr(binding, "mla_decode_tree_" + fmt)(q, qr, cache, table, ints(lens), parents.cuda(), SCALE,
                                                          workspace=ws)
    assert binding.mla_get_status(ws) == 0
    for b in range(len(lens)):
        for i in range(t):
            see = torch.as_tensor(expanded.tree_sees(parents[b].tolist(), t, i, lens[b] - t), device="cuda")
            k = rows[see + sum(lens[:b])].double()
            x = torch.cat([q[b, i], qr[b, i]], -1).double()
            if fmt.endswith("v41"):
                x[:, 448:512] = 0
            s = x @ k.T * SCALE
            p = torch.softmax(s, -1)
            ref, mag = p @ k[:, :512], p @ k[:, :512].abs()
            err = (out[b, i].double() - ref).abs()
            assert bool((err <= (2.0 ** -8 + 2.0 ** -9) * mag + 2.0 ** -8 * ref.abs()).all()), (b, i, float(err.max()))
            assert float((lse[b, i].double() - torch.logsumexp(s, -1)).abs().max()) <= 1e-3, (b, i)
    return rows


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,t", [([50, 200], 6), ([300], 1), ([1100], 3)])
def test_a_query_beyond_f16(cuda_device, fmt, lens, t):
    def prepare(c, q):
        c[:, 7] = 0                                  # what the large value meets
        q[0, t // 2, 5, 7] = 1e5

    run(fmt, lens, t, 5 + t, prepare)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,t", [([50, 200], 6), ([300], 1), ([1100], 3)])
def test_cached_values_beyond_f16(cuda_device, fmt, lens, t):
    def prepare(c, q):
        c[3, 32:64] *= 2.0 ** 20                     # one token's; a scale byte past the f16 pass's range
        q[..., 32:64] = 0

    rows = run(fmt, lens, t, 15 + t, prepare)
    assert float(rows[3, 32:64].float().abs().max()) > 65504
