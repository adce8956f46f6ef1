"""Decode of a drafted tree on the GPU against the float64 oracle.

Bounds: those of the dense decode's tests (max|out - ref| <= 1e-2 * max|ref|:
P is rounded to bf16, the result once more, 2^-8 each relative to sums of
|values| that stay below max|ref| + noise; max|lse - ref| <= 1e-3), and bit
equality where two calls must compute the same thing.
"""
import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from mla_latent_kv_05_gb300 import inputs as gen
from oracle import expanded, mla_oracle

pytestmark = pytest.mark.gpu

ENTRY = {"bf16": "bf16", "fp8": "fp8", "fp4": "fp4", "fp8v41": "fp8_v41", "fp4v41": "fp4_v41"}


def chain(b, t):
    return torch.arange(-1, t - 1, dtype=torch.int32).expand(b, t).contiguous()


def random_tree(b, t, seed):
    rng = np.random.default_rng(seed)
    return torch.tensor([[int(rng.integers(-1, i)) if i else -1 for i in range(t)] for _ in range(b)], dtype=torch.int32)


def run(inp, parents, n_nodes=None, ws=None, **kw):
    fn = getattr(binding, "mla_decode_tree_" + ENTRY[inp.kv_dtype])
    own = ws is None
    if own:
        ws = binding.alloc_workspace_tree(inp.batch, inp.sq)
    out, lse = fn(inp.q_absorbed.cuda(), inp.q_rope.cuda(), inp.kv_cache.cuda(), inp.block_table.cuda(),
                  inp.seq_lens.cuda(), parents.cuda(), inp.scale,
                  n_nodes=None if n_nodes is None else torch.tensor(n_nodes, dtype=torch.int32, device="cuda"),
                  workspace=ws, **kw)
    if own:
        assert binding.mla_get_status(ws) == 0
    return out, lse


def reference(inp, parents, n_nodes=None, rows_only=None):
    raw = inp.kv_cache.double().numpy() if inp.kv_dtype == "bf16" else inp.kv_cache.numpy()
    rows = mla_oracle.cache_rows(raw, inp.kv_dtype)
    out = np.zeros((inp.batch, inp.sq, 128, 512))
    lse = np.full((inp.batch, inp.sq, 128), -np.inf)
    for b in range(inp.batch):
        n = inp.sq if n_nodes is None else n_nodes[b]
        seq = int(inp.seq_lens[b])
        g = mla_oracle.gather_rows(rows, inp.block_table[b].numpy(), seq)
        for i in range(inp.sq):
            if rows_only is not None and (b, i) not in rows_only:
                continue
            see = expanded.tree_sees(parents[b].tolist(), n, i, seq - n)
            q = inp.q_absorbed[b, i].double().numpy().copy()
            if inp.kv_dtype.endswith("v41"):
                q[:, 448:] = 0
            if see.size:
                out[b, i], lse[b, i] = mla_oracle.attend_latent(q, inp.q_rope[b, i].double().numpy(), g[see], inp.scale)
    return out, lse


def check(out, lse, ref, rl, rows_only=None):
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(got.shape[0]):
        for i in range(got.shape[1]):
            if rows_only is not None and (b, i) not in rows_only:
                continue
            if np.isneginf(rl[b, i]).all():
                assert (got[b, i] == 0).all() and np.isneginf(gl[b, i]).all(), (b, i)
                continue
            assert np.abs(got[b, i] - ref[b, i]).max() <= 1e-2 * np.abs(ref[b, i]).max(), (b, i)
            assert np.abs(gl[b, i] - rl[b, i]).max() <= 1e-3, (b, i)


# contexts such that the drafted tokens start, end and straddle half pages, pages and score tiles
@pytest.mark.parametrize("t,lens", [(1, [1, 64, 300]), (5, [5, 6, 64, 69, 97, 130]), (8, [40, 1000]), (33, [33, 96, 128]),
                                    (64, [64, 65, 127, 161, 400]), (17, [2500])])
def test_random_trees(cuda_device, t, lens):
    inp = gen.make_inputs(len(lens), t, lens, seed=sum(lens) + t)
    parents = random_tree(len(lens), t, t)
    check(*run(inp, parents), *reference(inp, parents))


@pytest.mark.parametrize("fmt", ["fp8", "fp4", "fp8v41", "fp4v41"])
@pytest.mark.parametrize("t,lens", [(7, [7, 70, 260]), (40, [100, 641])])
def test_quantised_caches(cuda_device, fmt, t, lens):
    inp = gen.make_inputs(len(lens), t, lens, kv_dtype=fmt, seed=3 * t + len(fmt))
    parents = random_tree(len(lens), t, t + 1)
    check(*run(inp, parents), *reference(inp, parents))


def test_exact_pass_of_a_quantised_cache(cuda_device):
    # a query beyond f16 sends the call to the pass with bf16 operands
    inp = gen.make_inputs(2, 6, [50, 200], kv_dtype="fp8", seed=5)
    inp.q_absorbed[0, 2, 5, 7] = 1e5
    parents = random_tree(2, 6, 9)
    rows = [(b, i) for b in range(2) for i in range(6) if (b, i) != (0, 2)]
    check(*run(inp, parents), *reference(inp, parents), rows_only=rows)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_a_chain_is_the_causal_decode(cuda_device, fmt):
    inp = gen.make_inputs(3, 4, [4, 130, 700], kv_dtype=fmt, seed=6)
    out, lse = run(inp, chain(3, 4))
    fn = binding.mla_decode_bf16 if fmt == "bf16" else binding.mla_decode_fp8
    want, wl = fn(inp.q_absorbed.cuda(), inp.q_rope.cuda(), inp.kv_cache.cuda(), inp.block_table.cuda(),
                  inp.seq_lens.cuda(), inp.scale)
    # the same sums cut at other places: each side is within 1e-2 / 1e-3 of the
    # exact values, and this close to the other
    assert float((out.float() - want.float()).abs().max()) <= 2e-2 * float(want.float().abs().max())
    assert float((lse - wl).abs().max()) <= 2e-3


def test_fewer_nodes_than_the_call_holds(cuda_device):
    inp = gen.make_inputs(5, 9, [9, 20, 64, 300, 0], seed=7)
    n = [9, 1, 0, 6, 0]
    parents = random_tree(5, 9, 8)
    parents[1, 1:] = -7                                # behind n_nodes: not read
    out = torch.full((5, 9, 128, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 9, 128), float("nan"), device="cuda")
    got = run(inp, parents, n, out=out, lse=lse)
    check(*got, *reference(inp, parents, n))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_unseen_tokens_may_hold_anything(cuda_device, fmt):
    inp = gen.make_inputs(2, 12, [12 + 90, 12 + 250], kv_dtype=fmt, seed=8)
    parents = random_tree(2, 12, 10)
    want, wl = run(inp, parents)
    bad = {0: 3, 1: 5}                                 # one drafted token per sequence goes bad
    for b, a in bad.items():
        t = int(inp.seq_lens[b]) - 12 + a
        page = int(inp.block_table[b, t // 64])
        if fmt == "bf16":
            inp.kv_cache[page, t % 64] = float("nan")
        else:
            inp.kv_cache[page, t % 64] = 0x7F          # NaN codes
    got, gl = run(inp, parents)
    for b, a in bad.items():
        for i in range(12):
            up, sees = i, False
            while up >= 0:
                sees |= up == a
                up = int(parents[b, up])
            if sees:
                assert torch.isnan(got[b, i]).all()
            elif fmt == "bf16":
                assert torch.equal(got[b, i], want[b, i]) and torch.equal(gl[b, i], wl[b, i]), (b, i)
            else:
                torch.testing.assert_close(got[b, i].float(), want[b, i].float(), rtol=2e-2, atol=2e-2)


def test_many_rows_and_long_context_on_sampled_rows(cuda_device):
    lens = [3000 + 137 * b for b in range(10)]
    inp = gen.make_inputs(10, 48, lens, seed=9)
    parents = random_tree(10, 48, 11)
    rows = [(0, 0), (0, 47), (4, 20), (9, 47), (7, 3)]
    check(*run(inp, parents), *reference(inp, parents, rows_only=rows), rows_only=rows)


def test_wrong_numbers_are_recorded(cuda_device):
    inp = gen.make_inputs(3, 5, [30, 70, 100], seed=10)
    parents = random_tree(3, 5, 12)
    ws = binding.alloc_workspace_tree(3, 5)

    for bad in (3, 7, -2):                             # itself, a later node, below -1
        p = parents.clone()
        p[1, 3] = bad
        out, lse = run(inp, p, ws=ws)
        assert binding.mla_get_status(ws) == -8
        check(out, lse, *reference(inp, _ended(p)))
    for n in ([5, 6, 5], [5, -1, 5]):
        out, lse = run(inp, parents, n, ws=ws)
        assert binding.mla_get_status(ws) == -7
        assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())
    short = gen.make_inputs(3, 5, [30, 70, 100], seed=10)
    short.seq_lens[1] = 4
    out, lse = run(short, parents, ws=ws)
    assert binding.mla_get_status(ws) == -7
    assert bool((out[1] == 0).all())
    short.seq_lens[1] = short.max_pages * 64 + 1
    out, lse = run(short, parents, ws=ws)
    assert binding.mla_get_status(ws) == -7
    assert bool((out[1] == 0).all())
    paged = gen.make_inputs(3, 5, [30, 70, 100], seed=10)
    paged.block_table[2, 0] = paged.num_pages
    run(paged, parents, ws=ws)
    assert binding.mla_get_status(ws) == -5


def _ended(p):
    """A path ends at a parent outside [-1, its index)."""
    i = torch.arange(p.shape[1], dtype=torch.int32)
    return torch.where((p < -1) | (p >= i), torch.full_like(p, -1), p)


def test_captured_graph_with_new_trees(cuda_device):
    inp = gen.make_inputs(4, 10, [50, 300, 10, 129], seed=11)
    trees = [random_tree(4, 10, s) for s in (1, 2)]
    want = [run(inp, t) for t in trees]
    ws = binding.alloc_workspace_tree(4, 10)
    q, qr, kv, bt, sl = (x.cuda() for x in (inp.q_absorbed, inp.q_rope, inp.kv_cache, inp.block_table, inp.seq_lens))
    par = trees[0].cuda()
    out, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])

    def call():
        binding.mla_decode_tree_bf16(q, qr, kv, bt, sl, par, inp.scale, out=out, lse=lse, workspace=ws)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in (1, 0, 1):
        par.copy_(trees[k])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])
    assert binding.mla_get_status(ws) == 0


def test_prompt_chunk_draft_and_decode_together(cuda_device):
    """As a serving loop uses them: a prompt goes through expand and prefill
    and into the cache, a second chunk attends over the gathered context, a
    drafted tree is appended and verified by tree decode; the absorbed results
    go through W^UV.  Everything is checked against un-absorbed float64
    attention over the bf16 latents."""
    g = torch.Generator().manual_seed(21)

    def r(*shape, s=1.0):
        return (torch.randn(shape, generator=g) * s).to(torch.bfloat16).cuda()

    scale = 1.0 / 192 ** 0.5
    w_uk, w_uv = r(128, 128, 512, s=512 ** -0.5), r(128, 128, 512, s=512 ** -0.5)
    chunks, t = [70, 45], 6
    total = sum(chunks) + t
    c, kr = r(total, 512), r(total, 64)
    q_nope, q_rope = r(total, 128, 128), r(total, 128, 64)
    parents = torch.tensor([[-1, 0, 0, 1, -1, 4]], dtype=torch.int32, device="cuda")
    cache = torch.zeros((4, 64, 576), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")

    def ints(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    outs, lo = [], 0
    for n in chunks:
        hi = lo + n
        binding.mla_cache_append_bf16(c[lo:hi], kr[lo:hi], cache, table, ints(hi), ints(0, n))
        rows = binding.mla_cache_gather_bf16(cache, table, ints(hi), ints(0, hi), hi)
        k, v = binding.mla_expand_kv(rows[:, :512], w_uk, w_uv)
        outs.append(binding.mla_prefill_bf16(q_nope[lo:hi], q_rope[lo:hi], k, rows[:, 512:], v, ints(0, n), ints(0, hi),
                                             scale)[0])
        lo = hi
    binding.mla_cache_append_bf16(c[lo:], kr[lo:], cache, table, ints(total), ints(0, t))
    q_abs = torch.einsum("nhd,hdc->nhc", q_nope[lo:].float(), w_uk.float()).to(torch.bfloat16)[None].contiguous()
    lat, _ = binding.mla_decode_tree_bf16(q_abs, q_rope[lo:][None].contiguous(), cache, table, ints(total), parents, scale)
    outs.append(binding.mla_up_project_wuv(lat, w_uv)[0])
    got = torch.cat(outs).double()

    see = torch.ones((total, total), dtype=torch.bool, device="cuda").tril()
    for i in range(t):
        ok = expanded.tree_sees(parents[0].tolist(), t, i, lo)
        see[lo + i] = False
        see[lo + i, torch.tensor(ok, device="cuda")] = True
    k = torch.einsum("nc,hdc->hnd", c.double(), w_uk.double())
    v = torch.einsum("nc,hdc->hnd", c.double(), w_uv.double())
    s = scale * (torch.einsum("nhd,hmd->hnm", q_nope.double(), k) + torch.einsum("nhd,md->hnm", q_rope.double(), kr.double()))
    p = torch.softmax(s.masked_fill(~see, -torch.inf), -1)
    ref = torch.einsum("hnm,hmd->nhd", p, v)
    # roundings on the way: the expanded keys or the absorbed query (2^-8 of
    # values whose products sum to |s| ~ 1: under 1e-2 on a score, so under
    # 1e-2 of sum p|v|), P, V or the latent, and the result (2^-8 each)
    mag = torch.einsum("hnm,hmd->nhd", p, v.abs())
    assert bool(((got - ref).abs() <= (1e-2 + 3 * 2.0 ** -8) * mag + 2.0 ** -8 * ref.abs()).all())


@pytest.mark.parametrize("length", [40, 5000])
def test_a_nan_query_gives_nan_rows_only_for_itself(cuda_device, length):
    # 5000 tokens on one sequence: rows are split over several parts and merged
    inp = gen.make_inputs(1, 4, [length], seed=13)
    inp.q_absorbed[0, 2, 5] = float("nan")
    out, lse = run(inp, chain(1, 4))
    bad = torch.zeros((4, 128), dtype=torch.bool, device="cuda")
    bad[2, 5] = True
    assert torch.equal(torch.isnan(out[0]).all(-1), bad) and torch.equal(torch.isnan(out[0]).any(-1), bad)
    assert torch.equal(torch.isnan(lse[0]), bad)


def test_many_sequences_whose_rows_exceed_the_cache(cuda_device):
    # several rows a pair, uneven lengths, an empty sequence and one without nodes
    lens = [700 + 61 * b for b in range(40)]
    lens[7], lens[11] = 6, 0
    inp = gen.make_inputs(40, 6, lens, seed=14)
    n = [6] * 40
    n[11], n[20] = 0, 0
    parents = random_tree(40, 6, 15)
    rows = [(b, i) for b in (0, 7, 11, 20, 39) for i in (0, 5)]
    check(*run(inp, parents, n), *reference(inp, parents, n, rows_only=rows), rows_only=rows)


def test_the_most_sequences_a_call_takes(cuda_device):
    batch = 1 << 16
    q = torch.zeros((batch, 1, 128, 512), dtype=torch.bfloat16, device="cuda")
    qr = torch.zeros((batch, 1, 128, 64), dtype=torch.bfloat16, device="cuda")
    cache = torch.arange(4 * 64, device="cuda").to(torch.bfloat16)[:, None].expand(256, 576).reshape(4, 64, 576).contiguous()
    b = torch.arange(batch, device="cuda")
    table = (b % 4).to(torch.int32)[:, None].contiguous()
    lens = (b % 65).to(torch.int32)                       # a node of an empty sequence is none
    nodes = (lens > 0).to(torch.int32)
    out, lse = binding.mla_decode_tree_bf16(q, qr, cache, table, lens, torch.full((batch, 1), -1, dtype=torch.int32, device="cuda"),
                                            192 ** -0.5, n_nodes=nodes)
    # all scores are 0: the mean of tokens 64 p .. 64 p + len - 1 (below 256), rounded once
    mean = torch.where(lens > 0, (64 * table[:, 0] + (lens - 1) / 2).float(), torch.zeros((), device="cuda"))
    assert float((out[:, 0, ::31, ::73].float() - mean[:, None, None]).abs().max()) <= 2.0 ** -8 * 256
    want = torch.log(lens.float())
    assert torch.equal(torch.isneginf(lse[:, 0, 5]), lens == 0)
    assert float((lse[:, 0, 5] - want)[lens > 0].abs().max()) <= 1e-3
