"""Addresses past 4 GiB and the largest counts: caches, packed queries, keys and
outputs whose last rows lie beyond 32 bits of bytes, and of values, give the bits
of the same call over small tensors; 65,536 sequences in one prefill."""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from test_gpu_tree import random_tree

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
WIDTH = binding._ROW_WIDTH


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("fmt,pages", [("bf16", 60_000), ("fp8", 115_000), ("fp4_v41", 235_000)])
def test_pages_at_the_end_of_a_large_cache(cuda_device, fmt, pages):
    lens, t = [70, 300, 129], 6
    g = torch.Generator().manual_seed(pages)
    c, kr = (torch.randn((sum(lens), m), generator=g).to(torch.bfloat16).cuda() for m in (512, 64))
    q, qr = (torch.randn((3, t, 128, m), generator=g).to(torch.bfloat16).cuda() for m in (512, 64))
    parents, cu = random_tree(3, t, 2).cuda(), ints([0, 70, 370, 499])
    kind = torch.bfloat16 if fmt == "bf16" else torch.uint8
    got = []
    for n in (20, pages):
        cache = torch.empty((n, 64, WIDTH[fmt]), dtype=kind, device="cuda")
        assert n == 20 or cache.numel() * cache.element_size() > 1 << 32
        table = torch.full((3, 5), -1, dtype=torch.int32)
        at = n - 1
        for b, s in enumerate(lens):
            for k in range(-(-s // 64)):
                table[b, k] = at
                at -= 1
        table, sl = table.cuda(), ints(lens)
        getattr(binding, "mla_cache_append_" + fmt)(c, kr, cache, table, sl, cu)
        rows = getattr(binding, "mla_cache_gather_" + fmt)(cache, table, sl, cu, sum(lens))
        ws = binding.alloc_workspace_tree(3, t, max_pages=0 if fmt == "bf16" else 5)
        tree = getattr(binding, "mla_decode_tree_" + fmt)(q, qr, cache, table, sl, parents, SCALE, workspace=ws)
        assert binding.mla_get_status(ws) == 0
        got.append((rows,) + tree)
        del cache
    for a, b in zip(*got):
        assert torch.equal(a, b)
    torch.cuda.empty_cache()


def test_a_step_of_many_sequences(cuda_device):
    batch = 60_000
    g = torch.Generator().manual_seed(1)
    c, kr = (torch.randn((batch, m), generator=g).to(torch.bfloat16).cuda() for m in (512, 64))
    cache = torch.zeros((batch, 64, 576), dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(batch, generator=g).to(torch.int32)[:, None].cuda()
    lens = torch.randint(1, 65, (batch,), generator=g).to(torch.int32).cuda()
    cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    binding.mla_cache_append_bf16(c, kr, cache, table, lens, cu)
    got = cache[table[:, 0].long(), lens.long() - 1]
    assert torch.equal(got, torch.cat([c, kr], 1))
    assert int((cache != 0).any(-1).sum()) == batch
    assert torch.equal(binding.mla_cache_gather_bf16(cache, table, lens, cu, batch), got)
    del cache
    torch.cuda.empty_cache()


def test_prefill_rows_at_the_end_of_large_tensors(cuda_device):
    n, used = 140_000, 300                       # 2.3 G values in each of the keys, values and results
    g = torch.Generator().manual_seed(2)
    d = [torch.randn((used,) + s, generator=g).to(torch.bfloat16).cuda() for s in ((128, 128), (128, 64), (128, 128), (64,), (128, 128))]
    cu = ints([0, 120, used])
    want, wl = binding.mla_prefill_bf16(*d, cu, cu, SCALE)
    big = []
    for x in d:
        b = torch.empty((n,) + tuple(x.shape[1:]), dtype=torch.bfloat16, device="cuda")
        b[n - used:] = x
        big.append(b)
    at = cu + (n - used)
    ws = binding.alloc_workspace_prefill(2, n)
    out, lse = binding.mla_prefill_bf16(*big, at, at, SCALE, workspace=ws)
    assert binding.mla_get_status(ws) == 0
    assert torch.equal(out[n - used:], want) and torch.equal(lse[n - used:], wl)
    del big, out
    torch.cuda.empty_cache()


def test_expansion_of_many_rows(cuda_device):
    n = 140_000
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = torch.randn((n, 512), generator=g, device="cuda").to(torch.bfloat16)
    w = [(torch.randn((128, 128, 512), generator=g, device="cuda") * 512 ** -0.5).to(torch.bfloat16) for _ in range(2)]
    k, v = binding.mla_expand_kv(rows, *w)
    for lo in (0, 131_000, n - 400):
        a, b = binding.mla_expand_kv(rows[lo:lo + 400], *w)
        assert torch.equal(k[lo:lo + 400], a) and torch.equal(v[lo:lo + 400], b)
    del k, v
    torch.cuda.empty_cache()


def test_the_most_sequences_a_prefill_takes(cuda_device):
    # one query and one key each, every third without a key: the result is the
    # key's value (a weight of one), the lse its score
    batch = 1 << 16
    g = torch.Generator(device="cuda").manual_seed(4)

    def r(*s):
        return torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)

    has = torch.arange(batch, device="cuda") % 3 != 2
    nk = int(has.sum())
    q, qr, k, kr, v = r(batch, 128, 128), r(batch, 128, 64), r(nk, 128, 128), r(nk, 64), r(nk, 128, 128)
    cu_q = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    cu_k = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), has.cumsum(0)]).to(torch.int32)
    ws = binding.alloc_workspace_prefill(batch, batch)
    out, lse = binding.mla_prefill_bf16(q, qr, k, kr, v, cu_q, cu_k, SCALE, workspace=ws)
    assert binding.mla_get_status(ws) == 0
    assert torch.equal(out[has], v)
    assert bool((out[~has] == 0).all()) and bool(torch.isneginf(lse[~has]).all())
    for lo in range(0, nk, 1 << 13):
        at = torch.nonzero(has)[lo:lo + (1 << 13), 0]
        s = (q[at].double() * k[lo:lo + (1 << 13)].double()).sum(-1) + (qr[at].double() * kr[lo:lo + (1 << 13), None].double()).sum(-1)
        # 192 products in fp32: 192 * 2^-24 of scale sum|q||k| < 30
        assert float((lse[at].double() - SCALE * s).abs().max()) <= 1e-3
    del out, v, k, q
    torch.cuda.empty_cache()
