"""Cache rows on the GPU: append against the float64 encoder (bytes equal),
gather against the float64 decoders (the same bf16 value), the values where
the scale or a code sits at an edge, strided sources, rows that must stay as
they were, bad pages and lengths, other streams and captured graphs."""
import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from oracle import fp4_codec, fp8_codec, row_codec

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "fp8", "fp4", "fp8_v41", "fp4_v41"]
WIDTH = {"bf16": 576, "fp8": 594, "fp4": 324, "fp8_v41": 528, "fp4_v41": 288}
DECODE = {"fp8": fp8_codec.dequant_rows, "fp8_v41": fp8_codec.dequant_rows_v41, "fp4": fp4_codec.dequant_rows,
          "fp4_v41": fp4_codec.dequant_rows_v41}


def layout(new, ctx, seed, pool_extra=3):
    """block table, seq_lens, cu_rows and the cache slot of every packed row."""
    rng = np.random.default_rng(seed)
    lens = [a + c for a, c in zip(new, ctx)]
    need = [-(-s // 64) for s in lens]
    pool = sum(need) + pool_extra
    perm = rng.permutation(pool)
    table = np.full((len(new), max(1, max(need))), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    slots = [table[b, t // 64] * 64 + t % 64 for b in range(len(new)) for t in range(ctx[b], lens[b])]
    return table, np.array(lens, np.int32), cu, np.array(slots, np.int64), pool


def fresh_cache(fmt, pool, seed=0):
    g = torch.Generator().manual_seed(seed)
    raw = torch.randint(0, 256, (pool, 64, WIDTH[fmt] * (2 if fmt == "bf16" else 1)), generator=g).to(torch.uint8)
    return raw.view(torch.bfloat16) if fmt == "bf16" else raw


def values(n, seed):
    g = torch.Generator().manual_seed(seed)
    c = torch.randn((n, 512), generator=g) * torch.exp2(torch.randint(-6, 6, (n, 1), generator=g))
    r = torch.randn((n, 64), generator=g)
    return c.to(torch.bfloat16), r.to(torch.bfloat16)


def expected_bytes(fmt, c, r):
    if fmt == "bf16":
        return torch.cat([c, r], -1).view(torch.uint8).numpy()
    return row_codec.encode_rows(c.double().numpy(), r.double().numpy(), fmt)


def append(fmt, c, r, cache, table, lens, cu, ws=None, stream=None):
    return getattr(binding, "mla_cache_append_" + fmt)(c, r, cache, table, lens, cu, workspace=ws, stream=stream)


def gather(fmt, cache, table, lens, cu, n, **kw):
    return getattr(binding, "mla_cache_gather_" + fmt)(cache, table, lens, cu, n, **kw)


def dev(*xs):
    return [torch.as_tensor(x).cuda() for x in xs]


def raw_of(cache):
    return cache.cpu().view(torch.uint8).reshape(-1, cache.shape[-1] * cache.element_size()).numpy()


CASES = [([1], [0]), ([1] * 33, list(range(33))), ([5, 0, 64, 65, 1], [0, 7, 0, 63, 128]), ([130, 3], [61, 4000]),
         ([0, 0, 2], [5, 0, 0])]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("new,ctx", CASES)
def test_append_writes_the_rows_and_nothing_else(cuda_device, fmt, new, ctx):
    table, lens, cu, slots, pool = layout(new, ctx, 5)
    c, r = values(sum(new), 11)
    cache = fresh_cache(fmt, pool)
    want = raw_of(cache).copy()
    want[slots] = expected_bytes(fmt, c, r)
    d = cache.cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert append(fmt, *dev(c, r), d, *dev(table, lens, cu), ws=ws) is d
    assert binding.mla_get_status(ws) == 0
    np.testing.assert_array_equal(raw_of(d), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("new,ctx", CASES)
def test_gather_reads_the_rows_values(cuda_device, fmt, new, ctx):
    table, lens, cu, slots, pool = layout(new, ctx, 6)
    cache = fresh_cache(fmt, pool, 1)
    if fmt != "bf16":      # any byte is a code; keep the scales where bf16 holds the product, and one NaN scale
        cache[..., -1] = 255
        cache[..., -2] = 3
    raw = raw_of(cache)[slots]
    n = sum(new)
    out = torch.full((n + 2, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    gather(fmt, cache.cuda(), *dev(table, lens, cu), n + 2, out=out, workspace=ws)
    assert binding.mla_get_status(ws) == 0
    got = out.cpu()
    assert torch.all(got[n:] == 7.0)                       # behind the last sequence: as it was
    if fmt == "bf16":
        np.testing.assert_array_equal(got[:n].contiguous().view(torch.uint8).numpy().reshape(n, -1), raw)
        return
    with np.errstate(over="ignore"):
        want = torch.from_numpy(DECODE[fmt](raw)).to(torch.bfloat16)
    a, b = got[:n].float(), want.float()
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(torch.nan_to_num(a, nan=0.0, posinf=None, neginf=None), torch.nan_to_num(b, nan=0.0))


@pytest.mark.parametrize("fmt", FORMATS[1:])
def test_scales_and_codes_at_their_edges(cuda_device, fmt):
    # one group kind per row: zeros, the borders of the scale choice, ties of
    # the codes, the largest and smallest bf16 values, infinities and NaNs
    top = 448.0 if fmt.startswith("fp8") else 6.0
    kinds = []
    for v in (0.0, top, top * (1 + 2 ** -7), top / 2, 3.3895e38, -3.3895e38, 2.0 ** -126, 2.0 ** -133, 9.2e-41,
              float("inf"), float("-inf"), float("nan")):
        x = torch.zeros(576)
        x[::16] = v
        x[5::16] = v / 3 if np.isfinite(v) else 1.0
        kinds.append(x)
    ties = torch.zeros(576)
    grid = torch.tensor([448.0, 17, 19, 21, 25, 2.0 ** -10, 3 * 2.0 ** -10, 5 * 2.0 ** -10, 0.0, -0.0, -17, 1.0625, 1.1875,
                         240, 232, 248]) if top == 448.0 else \
        torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -5.0, 0.2578125, 0.24902, 0.0, -0.0])
    ties[:] = grid.repeat(36)
    kinds.append(ties)
    x = torch.stack(kinds).to(torch.bfloat16)
    c, r = x[:, :512].contiguous(), x[:, 512:].contiguous()
    n = x.shape[0]
    table, lens, cu, slots, pool = layout([n], [0], 3)
    d = fresh_cache(fmt, pool).cuda()
    append(fmt, *dev(c, r), d, *dev(table, lens, cu))
    got = raw_of(d)[slots]
    np.testing.assert_array_equal(got, expected_bytes(fmt, c, r))
    back = gather(fmt, d, *dev(table, lens, cu), n).float().cpu()
    latent = 448 if fmt.endswith("v41") else 512
    bad = torch.tensor([not bool(torch.isfinite(k).all()) for k in kinds])
    assert torch.isnan(back[bad][:, :latent]).all()        # a non-finite value reads back as NaN, its group with it
    assert torch.isfinite(back[~bad]).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4_v41"])
def test_strided_sources(cuda_device, fmt):
    new, ctx = [70, 9], [3, 200]
    table, lens, cu, slots, pool = layout(new, ctx, 8)
    c, r = values(79, 12)
    both = torch.zeros((79, 3, 584), dtype=torch.bfloat16, device="cuda")
    both[:, 1, :512] = c.cuda()
    both[:, 1, 512:576] = r.cuda()
    d = fresh_cache(fmt, pool).cuda()
    append(fmt, both[:, 1, :512], both[:, 1, 512:576], d, *dev(table, lens, cu))
    np.testing.assert_array_equal(raw_of(d)[slots], expected_bytes(fmt, c, r))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_rows_outside_the_cache_are_recorded_and_left(cuda_device, fmt):
    new, ctx = [4, 5, 6], [60, 0, 10]
    table, lens, cu, slots, pool = layout(new, ctx, 9)
    c, r = values(15, 13)
    want_rows = expected_bytes(fmt, c, r)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for kind, code in (("page", -5), ("page high", -5), ("short", -7), ("long", -7)):
        t, s = table.copy(), lens.copy()
        lost = set(range(4, 9))                            # the second sequence's rows
        if kind == "page":
            t[1, 0] = -1
        elif kind == "page high":
            t[1, 0] = pool
        elif kind == "short":
            s[1] = 2                                       # fewer tokens than rows: its first three rows have none
            lost = set(range(4, 7))
        else:
            s[1] = t.shape[1] * 64 + 2                     # its last two tokens lie past the table
            lost = {7, 8} | set(range(4, 7))
            t[1, 1:] = -1
            t[1, -1] = -1
        cache = fresh_cache(fmt, pool)
        before = raw_of(cache).copy()
        d = cache.cuda()
        append(fmt, *dev(c, r), d, *dev(t, s, cu), ws=ws)
        st = binding.mla_get_status(ws)
        assert st in (-5, -7) if kind == "long" else st == code, kind
        after = raw_of(d)
        kept = [i for i in range(15) if i not in lost and not 4 <= i < 9]
        np.testing.assert_array_equal(after[slots[kept]], want_rows[kept])
        if kind == "short":
            np.testing.assert_array_equal(after[slots[[4, 5]]], want_rows[[7, 8]])   # tokens 0 and 1 of the sequence
        out = gather(fmt, d, *dev(t, s, cu), 15, workspace=ws).cpu()
        assert binding.mla_get_status(ws) in (-5, -7)
        assert torch.all(out[sorted(lost)] == 0), kind
        changed = np.nonzero((after != before).any(1))[0]
        assert set(changed) <= set(slots.tolist())


def test_many_sequences_and_a_captured_graph(cuda_device):
    # more sequences than one search round covers; replayed with new lengths
    B = 1500
    new = [1 + (i % 3) for i in range(B)]
    ctx = [i % 70 for i in range(B)]
    table, lens, cu, slots, pool = layout(new, ctx, 10)
    c, r = values(sum(new), 14)
    dc, dr = dev(c, r)
    dt, dl, du = dev(table, lens, cu)
    d = fresh_cache("fp8", pool).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.empty((sum(new), 576), dtype=torch.bfloat16, device="cuda")
    append("fp8", dc, dr, d, dt, dl, du, ws=ws)
    np.testing.assert_array_equal(raw_of(d)[slots], expected_bytes("fp8", c, r))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        append("fp8", dc, dr, d, dt, dl, du, ws=ws)
        gather("fp8", d, dt, dl, du, sum(new), out=out, workspace=ws)
    c2, r2 = values(sum(new), 15)
    dc.copy_(c2)
    dr.copy_(r2)
    g.replay()
    torch.cuda.synchronize()
    assert binding.mla_get_status(ws) == 0
    rows = expected_bytes("fp8", c2, r2)
    np.testing.assert_array_equal(raw_of(d)[slots], rows)
    want = torch.from_numpy(fp8_codec.dequant_rows(rows)).to(torch.bfloat16)
    assert torch.equal(out.cpu(), want)


def test_another_stream(cuda_device):
    table, lens, cu, slots, pool = layout([300], [0], 20)
    c, r = values(300, 21)
    d = fresh_cache("fp4", pool).cuda()
    args = dev(c, r)
    idx = dev(table, lens, cu)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    append("fp4", *args, d, *idx, stream=s)
    s.synchronize()
    np.testing.assert_array_equal(raw_of(d)[slots], expected_bytes("fp4", c, r))
