"""Tree decode whose scores rise along the sequence, so that the reference
maximum of a head moves in tile after tile and its output is rescaled.

Three RoPE dimensions of the cached rows hold stairs of 64, 128 and 192 tokens a
step; a third of the heads reads each, the last few none.  A step is worth about
14.4 in log2 units, above the 12 that move the reference, and a step's tokens
weigh the same, so that both pages of a tile, and both halves of a head's
columns, count in the result.

Bound per element: P is rounded to bf16 (2^-8 of sum p|v|) and the result once
more (2^-8 of |out|).  The fp32 sums before the scale reach 5600, where a
rounding is worth at most 2^-11, 3.6e-5 once scaled; the RoPE products that come
after the stairs make 64 of them, 2.3e-3 in the worst order and 3e-4 as a random
walk, taken twice (numerator and denominator): 2^-9 of sum p|v|, and 1e-3 of the
lse.
"""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from test_gpu_tree import random_tree
from oracle import expanded

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
STEP = 10.0 / (SCALE * 8)       # 10 nats for a query value of 8


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def case(fmt, lens, t, seed):
    g = torch.Generator().manual_seed(seed)
    total = sum(lens)
    c = torch.randn((total, 512), generator=g).to(torch.bfloat16).cuda()
    kr = torch.randn((total, 64), generator=g)
    at = torch.cat([torch.arange(n) for n in lens])
    for d, width in enumerate((64, 128, 192)):
        kr[:, d] = torch.floor(at / width) * STEP
    kr = kr.to(torch.bfloat16).cuda()
    pages = -(-max(lens) // 64)
    table = torch.randperm(len(lens) * pages, generator=g).to(torch.int32).view(len(lens), pages).cuda()
    width = binding._ROW_WIDTH[fmt]
    cache = torch.zeros((len(lens) * pages, 64, width), device="cuda",
                        dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8)
    cu = ints([0] + [sum(lens[:b + 1]) for b in range(len(lens))])
    getattr(binding, "mla_cache_append_" + fmt)(c, kr, cache, table, ints(lens), cu)
    rows = getattr(binding, "mla_cache_gather_" + fmt)(cache, table, ints(lens), cu, total)
    q = torch.randn((len(lens), t, 128, 512), generator=g).to(torch.bfloat16).cuda()
    qr = torch.randn((len(lens), t, 128, 64), generator=g)
    for d in range(3):
        qr[..., d] = torch.where((torch.arange(128) % 3 == d) & (torch.arange(128) < 120), 8.0, 0.0)
    return q, qr.to(torch.bfloat16).cuda(), cache, table, rows


def check(out, lse, q, qr, rows, lens, parents, b, i, v41):
    t = parents.shape[1]
    lo = sum(lens[:b])
    see = torch.as_tensor(expanded.tree_sees(parents[b].tolist(), t, i, lens[b] - t), device="cuda") + lo
    k = rows[see].double()
    x = torch.cat([q[b, i], qr[b, i]], -1).double()
    if v41:
        x[:, 448:512] = 0
    s = x @ k.T * SCALE
    p = torch.softmax(s, -1)
    ref, mag = p @ k[:, :512], p @ k[:, :512].abs()
    err = (out[b, i].double() - ref).abs()
    assert bool((err <= (2.0 ** -8 + 2.0 ** -9) * mag + 2.0 ** -8 * ref.abs()).all()), (b, i, float(err.max()))
    assert float((lse[b, i].double() - torch.logsumexp(s, -1)).abs().max()) <= 1e-3, (b, i)


# one sequence in many parts; few rows, cut; rows that mostly stay whole.  The
# ends put the drafted tokens into the first page of a tile, the second and both.
CASES = [([1500], 3), ([2575, 2497], 9), ([700, 641, 770], 40), ([1100, 1090], 64)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4", "fp8_v41", "fp4_v41"])
@pytest.mark.parametrize("lens,t", CASES)
def test_references_that_move(cuda_device, fmt, lens, t):
    q, qr, cache, table, rows = case(fmt, lens, t, 7 * t + len(lens))
    parents = random_tree(len(lens), t, t + 3)
    ws = binding.alloc_workspace_tree(len(lens), t, max_pages=0 if fmt == "bf16" else table.shape[1])
    fn = getattr(binding, "mla_decode_tree_" + fmt)
    args = q, qr, cache, table, ints(lens), parents.cuda(), SCALE
    out, lse = fn(*args, workspace=ws)
    assert binding.mla_get_status(ws) == 0
    for b in range(len(lens)):
        for i in range(t):
            check(out, lse, q, qr, rows, lens, parents, b, i, fmt.endswith("v41"))
    for _ in range(20):                       # the same bits every time
        again, al = fn(*args, workspace=ws)
        assert torch.equal(again, out) and torch.equal(al, lse)
