"""Rotary positions and the rotating cache append on the GPU against float64 oracles.

Rotation: the products and their sum in fp32 are off by at most 3 * 2^-24 of |a| + |b| each (and the cosine and sine
by 2^-24 of theirs), together under 2^-21 (|a| + |b|) scale; the result is then rounded to bf16, at most half a step:
eight significant bits, so a step is 2^-7 of a binade's lower end and half of it 2^-8 of the value (plus that error).  Append: the cache holds the bytes of the exactly rotated values, encoded by the row oracle; positions below
2^18, where a float64 angle is known to 2^-35, so that the oracle and the kernel (2^-40) agree on the side of every
border unless a value lies within 2^-34 of one (one value in 10^8; the inputs are fixed).
"""
import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from oracle import rope, row_codec

pytestmark = pytest.mark.gpu

FORMATS = {"bf16": 576, "fp8": 594, "fp4": 324, "fp8_v41": 528, "fp4_v41": 288}


def normal(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


def check(y, x, pos, f, interleaved, scale=1.0, inverse=False):
    x = x.double().numpy()
    want = rope.rotate(x, pos, f, interleaved, scale, inverse)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    mag = np.abs(a) + np.abs(b)
    mag = np.repeat(mag, 2, -1) if interleaved else np.concatenate([mag, mag], -1)
    fp32 = 2.0 ** -21 * mag * abs(scale)
    got = y.double().cpu().numpy()
    assert (np.abs(got - want) <= fp32 + 2.0 ** -8 * (np.abs(want) + fp32)).all()


# ------------------------------------------------------------------ rotation
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rows,heads", [(1, 1), (1, 128), (3, 5), (63, 1), (65, 1), (64, 64), (200, 16), (130, 128),
                                        (1000, 65), (2049, 128), (5000, 1), (700, 33)])
def test_rotation(cuda_device, rows, heads, interleaved):
    g = torch.Generator().manual_seed(rows * 131 + heads)
    x, f = normal(g, rows, heads, 64), rope.frequencies(factor=40.0 if rows % 2 else 1.0)
    pos = torch.randint(0, 163840, (rows,), generator=g).to(torch.int32)
    t = binding.mla_rope_init(f, interleaved=interleaved)
    y = binding.mla_rope_bf16(x.cuda(), pos.cuda(), t)
    check(y, x, pos.numpy(), f, interleaved)
    z = binding.mla_rope_bf16(x.cuda(), pos.cuda(), t, inverse=True)
    check(z, x, pos.numpy(), f, interleaved, inverse=True)


def test_keys_without_a_head_dimension_and_the_scale(cuda_device):
    g = torch.Generator().manual_seed(5)
    x, f = normal(g, 77, 64), rope.frequencies()
    pos = torch.arange(77, dtype=torch.int32)
    y = binding.mla_rope_bf16(x.cuda(), pos.cuda(), binding.mla_rope_init(f, scale=1.3))
    assert y.shape == (77, 64)
    check(y, x, pos.numpy(), f, True, scale=np.float32(1.3))
    zero = binding.mla_rope_bf16(x.cuda(), torch.zeros(77, dtype=torch.int32).cuda(), binding.mla_rope_init(f))
    assert torch.equal(zero.cpu(), x)                     # position 0 turns nothing


def test_far_and_negative_positions(cuda_device):
    # angles from the table's own fractions of a turn, in integers
    g = torch.Generator().manual_seed(6)
    f = rope.frequencies()
    t = binding.mla_rope_init(f)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 1, 2 ** 30 + 12345, -987654321, 16777217], dtype=torch.int32)
    x = normal(g, 7, 2, 64)
    y = binding.mla_rope_bf16(x.cuda(), pos.cuda(), t).double().cpu().numpy()
    turns = np.array([[(int(p) * int(u) % 2 ** 64) / 2.0 ** 64 for u in t.turns] for p in pos])
    a, b = x.double().numpy()[..., 0::2], x.double().numpy()[..., 1::2]
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    bound = 2.0 ** -21 * (np.abs(a) + np.abs(b))
    for got, want in ((y[..., 0::2], a * c - b * s), (y[..., 1::2], a * s + b * c)):
        assert (np.abs(got - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()


@pytest.mark.parametrize("interleaved", [True, False])
def test_views_and_in_place(cuda_device, interleaved):
    g = torch.Generator().manual_seed(7)
    q, f = normal(g, 300, 128, 192), rope.frequencies()
    pos = torch.randint(0, 4096, (300,), generator=g).to(torch.int32)
    t = binding.mla_rope_init(f, interleaved=interleaved)
    dq = q.cuda()
    want = binding.mla_rope_bf16(dq[..., 128:].contiguous(), pos.cuda(), t)
    check(want, q[..., 128:], pos.numpy(), f, interleaved)
    assert torch.equal(binding.mla_rope_bf16(dq[..., 128:], pos.cuda(), t), want)
    part = dq[..., 128:]
    assert binding.mla_rope_bf16(part, pos.cuda(), t, out=part) is part
    assert torch.equal(part, want) and torch.equal(dq[..., :128].cpu(), q[..., :128])
    # heads before rows, into the same order
    y = torch.empty((128, 300, 64), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    x = q[..., 128:].transpose(0, 1).contiguous().cuda().transpose(0, 1)
    assert torch.equal(binding.mla_rope_bf16(x, pos.cuda(), t, out=y), want)


def test_every_other_row_and_a_single_head_of_many(cuda_device):
    g = torch.Generator().manual_seed(8)
    q, f = normal(g, 90, 6, 64).cuda(), rope.frequencies()
    pos = torch.randint(0, 4096, (45,), generator=g).to(torch.int32).cuda()
    t = binding.mla_rope_init(f)
    want = binding.mla_rope_bf16(q[::2].contiguous(), pos, t)
    assert torch.equal(binding.mla_rope_bf16(q[::2], pos, t), want)
    assert torch.equal(binding.mla_rope_bf16(q[::2, 3:4], pos, t), want[:, 3:4])
    assert torch.equal(binding.mla_rope_bf16(q[::2, 3], pos, t), want[:, 3])


def test_refusals_and_empty_calls(cuda_device):
    f = rope.frequencies()
    t = binding.mla_rope_init(f)
    x = torch.zeros((4, 8, 64), dtype=torch.bfloat16, device="cuda")
    p = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad, err in (((x.float(), p, t), TypeError), ((x, p.long(), t), TypeError), ((x, p[:3], t), ValueError),
                     ((x[..., :32], p, t), ValueError), ((x, p, f), TypeError), ((x.cpu(), p, t), ValueError),
                     ((x[:, :1].expand(4, 8, 64), p, t), ValueError), ((x[0, 0], p, t), ValueError)):
        with pytest.raises(err):
            binding.mla_rope_bf16(*bad)
    with pytest.raises(ValueError):
        binding.mla_rope_bf16(x, p, t, out=x[:3])
    with pytest.raises(ValueError):
        odd = torch.zeros(4 * 8 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 8, 64)
        binding.mla_rope_bf16(odd, p, t)
    assert binding.mla_rope_bf16(x[:0], p[:0], t).shape == (0, 8, 64)
    assert binding.mla_rope_bf16(x[:, :0], p, t).shape == (4, 0, 64)


# ------------------------------------------------------------------ append
class Cache:
    """Sequences with `new` rows each behind `ctx` cached tokens, over shuffled pages; `behind` more packed rows."""

    def __init__(self, new, ctx, seed, behind=0):
        self.g = torch.Generator().manual_seed(seed)
        self.new, self.lens = new, [n + c for n, c in zip(new, ctx)]
        self.n = sum(new)
        need = [(s + 63) // 64 for s in self.lens]
        self.pages = sum(need) + 3
        perm = torch.randperm(self.pages, generator=self.g).tolist()
        self.table = torch.full((len(new), max(max(need), 1)), -1, dtype=torch.int32)
        for b, k in enumerate(need):
            for i in range(k):
                self.table[b, i] = perm.pop()
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.c, self.r = normal(self.g, self.n + behind, 512), normal(self.g, self.n + behind, 64)
        self.tokens = np.concatenate([np.arange(s - n, s) for s, n in zip(self.lens, new)] or [[]]).astype(np.int64)
        self.slots = np.array([int(self.table[b, t // 64]) * 64 + t % 64
                               for b, (s, n) in enumerate(zip(self.lens, new)) for t in range(s - n, s)], dtype=np.int64)

    def empty(self, fmt):
        if fmt == "bf16":
            return torch.full((self.pages, 64, 576), 7.0, dtype=torch.bfloat16, device="cuda")
        return torch.full((self.pages, 64, FORMATS[fmt]), 0xA5, dtype=torch.uint8, device="cuda")

    def append(self, fmt, table, positions=None, cache=None, **kw):
        cache = self.empty(fmt) if cache is None else cache
        got = getattr(binding, "mla_cache_append_rope_" + fmt)(
            self.c.cuda(), self.r.cuda(), table, cache, self.table.cuda(),
            torch.tensor(self.lens, dtype=torch.int32).cuda(), self.cu.cuda(), positions=positions, **kw)
        assert got is cache
        return cache

    def want(self, fmt, f, interleaved, positions=None, scale=1.0):
        """The cache's rows, as bf16 or bytes; others as `empty` left them."""
        pos = self.tokens if positions is None else positions[:self.n]
        k = rope.rotate(self.r[:self.n].double().numpy(), pos, f, interleaved, scale)
        c = self.c[:self.n].double().numpy()
        full = self.empty(fmt).cpu().view(-1, FORMATS[fmt])
        if fmt == "bf16":
            # numpy rounds float64 to bf16 through torch: one rounding from float64 needs the odd last bit
            full[self.slots] = torch.cat([self.c[:self.n], round_bf16(k)], 1)
        else:
            full[self.slots] = torch.from_numpy(row_codec.encode_rows(c, k, fmt))
        return full.view(self.empty(fmt).shape)


def round_bf16(x):
    """float64 -> bf16, to nearest even, in one rounding."""
    m, e = np.frexp(x)
    return torch.from_numpy(np.ldexp(np.round(np.ldexp(m, 8)), e - 8)).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("new,ctx", [([1], [0]), ([1] * 9, [0, 63, 64, 65, 1000, 1, 2, 127, 128]), ([5, 0, 130, 1], [7, 9, 0, 300]),
                                     ([3000, 5300], [0, 1000])], ids=["one", "step", "ragged", "long"])
def test_append_writes_the_bytes_of_the_exactly_rotated_rows(cuda_device, fmt, interleaved, new, ctx):
    s = Cache(new, ctx, seed=len(new) + 10 * len(fmt))
    f = rope.frequencies(factor=40.0)
    t = binding.mla_rope_init(f, interleaved=interleaved)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    got = s.append(fmt, t, workspace=ws)
    assert torch.equal(got.cpu(), s.want(fmt, f, interleaved))
    assert binding.mla_get_status(ws) == 0


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_append_by_given_positions_and_a_scale(cuda_device, fmt):
    s = Cache([64, 33, 1], [500, 0, 9000], seed=3)
    f = rope.frequencies()
    pos = torch.randint(0, 163840, (s.n,), generator=s.g).to(torch.int32)
    got = s.append(fmt, binding.mla_rope_init(f, scale=0.75), positions=pos.cuda())
    assert torch.equal(got.cpu(), s.want(fmt, f, True, positions=pos.numpy(), scale=0.75))


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_position_zero_is_the_plain_append(cuda_device, fmt):
    s = Cache([300, 77], [0, 64], seed=4)
    zero = torch.zeros(s.n, dtype=torch.int32, device="cuda")
    got = s.append(fmt, binding.mla_rope_init(rope.frequencies()), positions=zero)
    want = getattr(binding, "mla_cache_append_" + fmt)(s.c.cuda(), s.r.cuda(), s.empty(fmt), s.table.cuda(),
                                                       torch.tensor(s.lens, dtype=torch.int32).cuda(), s.cu.cuda())
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_rows_behind_the_last_sequence_and_bad_rows_are_left_alone(cuda_device, fmt):
    s = Cache([10, 20], [0, 40], seed=5, behind=6)
    f = rope.frequencies()
    s.c[s.n:] = float("nan")
    pos = torch.arange(s.n + 6, dtype=torch.int32)
    got = s.append(fmt, binding.mla_rope_init(f), positions=pos.cuda())
    assert torch.equal(got.cpu(), s.want(fmt, f, True, positions=pos.numpy()))
    for bad, code in ((-5, -7), (10 ** 6, -7)):           # a length that does not hold the rows, or past the table
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        cache = s.empty(fmt)
        lens = torch.tensor([bad, s.lens[1]], dtype=torch.int32).cuda()
        getattr(binding, "mla_cache_append_rope_" + fmt)(s.c.cuda(), s.r.cuda(), binding.mla_rope_init(f), cache,
                                                         s.table.cuda(), lens, s.cu.cuda(), positions=pos.cuda(), workspace=ws)
        want, plain = s.want(fmt, f, True, positions=pos.numpy()), s.empty(fmt).cpu()
        want.view(-1, FORMATS[fmt])[s.slots[:10]] = plain.view(-1, FORMATS[fmt])[s.slots[:10]]
        assert torch.equal(cache.cpu(), want)
        assert binding.mla_get_status(ws) == code
    table = s.table.clone()
    table[1, 0] = s.pages                                 # tokens 40..63 of sequence 1 are on it
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cache = s.empty(fmt)
    getattr(binding, "mla_cache_append_rope_" + fmt)(s.c.cuda(), s.r.cuda(), binding.mla_rope_init(f), cache, table.cuda(),
                                                     torch.tensor(s.lens, dtype=torch.int32).cuda(), s.cu.cuda(),
                                                     positions=pos.cuda(), workspace=ws)
    want = s.want(fmt, f, True, positions=pos.numpy())
    want.view(-1, FORMATS[fmt])[s.slots[10:]] = s.empty(fmt).cpu().view(-1, FORMATS[fmt])[s.slots[10:]]
    assert torch.equal(cache.cpu(), want)
    assert binding.mla_get_status(ws) == -5


@pytest.mark.parametrize("fmt", list(FORMATS))
def test_values_that_are_not_finite_stay_in_their_group(cuda_device, fmt):
    s = Cache([6], [100], seed=6)
    s.r[1, 5], s.r[2, 40], s.r[4, 63] = float("inf"), float("nan"), float("-inf")
    s.c[5, 3] = float("inf")
    f = rope.frequencies()
    got = s.append(fmt, binding.mla_rope_init(f)).cpu()
    want = s.want(fmt, f, True)
    if fmt == "bf16":       # a NaN's bits are not defined
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    else:
        assert torch.equal(got, want)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_append_in_a_captured_graph_and_on_another_stream(cuda_device, fmt):
    s = Cache([40, 3], [5, 700], seed=7)
    f = rope.frequencies()
    t = binding.mla_rope_init(f)
    want = s.want(fmt, f, True)
    args = [x.cuda() for x in (s.c, s.r)], [s.table.cuda(), torch.tensor(s.lens, dtype=torch.int32).cuda(), s.cu.cuda()]
    ws, cache = torch.zeros(256, dtype=torch.uint8, device="cuda"), s.empty(fmt)
    fn = getattr(binding, "mla_cache_append_rope_" + fmt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fn(*args[0], t, cache, *args[1], workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(cache.cpu(), want)
    q = torch.randn((43, 128, 64), device="cuda").to(torch.bfloat16)
    pos = torch.arange(43, dtype=torch.int32, device="cuda")
    y = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    cache.copy_(s.empty(fmt))
    with torch.cuda.graph(graph):
        fn(*args[0], t, cache, *args[1], workspace=ws)
        binding.mla_rope_bf16(q, pos, t, out=y)
    t.scale = 0.0                                         # the calls copied the table
    graph.replay()
    torch.cuda.synchronize()
    t.scale = 1.0
    assert torch.equal(cache.cpu(), want)
    assert torch.equal(y, binding.mla_rope_bf16(q, pos, t))


@pytest.mark.parametrize("interleaved", [True, False])
def test_a_prompt_and_drafted_nodes_as_they_are_served(cuda_device, interleaved):
    """Rotation, append, gather, expansion, prefill and tree decode in a row, against the oracles on exactly rotated rows."""
    from oracle import expanded, mla_oracle
    g = torch.Generator().manual_seed(40)
    n, t, scale = 70, 4, 192 ** -0.5
    f = rope.frequencies(factor=40.0)
    table = binding.mla_rope_init(f, interleaved=interleaved)

    def bf16(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)

    def ints(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    c, kr, qn, qr, w_uk, w_uv = bf16(n + t, 512), bf16(n + t, 64), bf16(n, 128, 128), bf16(n, 128, 64), bf16(128, 128, 512), bf16(128, 128, 512)
    w_uk, w_uv = w_uk * 0.0625, w_uv * 0.0625          # (powers of two: exact)
    qa, qt, parents = bf16(1, t, 128, 512) * 0.25, bf16(1, t, 128, 64), [-1, 0, 0, 1]
    at = np.array([n, n + 1, n + 1, n + 2])            # a node's position is its depth's, not its place in the cache
    cache, pages = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda"), ints(1, 0)[None].contiguous()
    binding.mla_cache_append_rope_bf16(c[:n].cuda(), kr[:n].cuda(), table, cache, pages, ints(n), ints(0, n))
    q_rot = binding.mla_rope_bf16(qr.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"), table)
    rows = binding.mla_cache_gather_bf16(cache, pages, ints(n), ints(0, n), n)
    k, v = binding.mla_expand_kv(rows[:, :512], w_uk.cuda(), w_uv.cuda())
    out, lse = binding.mla_prefill_bf16(qn.cuda(), q_rot, k, rows[:, 512:], v, ints(0, n), ints(0, n), scale)
    exact_k = round_bf16(rope.rotate(kr[:n].double().numpy(), np.arange(n), f, interleaved))
    assert torch.equal(rows.cpu(), torch.cat([c[:n], exact_k], 1))
    for h in (0, 77):
        q = np.concatenate([qn[:, h].double().numpy(),
                            round_bf16(rope.rotate(qr[:, h].double().numpy(), np.arange(n), f, interleaved)).double().numpy()], 1)
        kk = np.concatenate([k[:, h].double().cpu().numpy(), exact_k.double().numpy()], 1)
        o, l, _ = expanded.attend(q, kk, v[:, h].double().cpu().numpy(), np.tril(np.ones((n, n), dtype=bool)), scale)
        assert np.abs(out[:, h].double().cpu().numpy() - o).max() <= 1e-2 * np.abs(o).max()
        assert np.abs(lse[:, h].double().cpu().numpy() - l).max() <= 1e-3
    binding.mla_cache_append_rope_bf16(c[n:].cuda(), kr[n:].cuda(), table, cache, pages, ints(n + t), ints(0, t), positions=ints(*at))
    qt_rot = binding.mla_rope_bf16(qt[0].cuda(), ints(*at), table)[None]
    to, tl = binding.mla_decode_tree_bf16(qa.cuda(), qt_rot, cache, pages, ints(n + t), ints(*parents)[None].contiguous(), scale)
    k_all = torch.cat([exact_k, round_bf16(rope.rotate(kr[n:].double().numpy(), at, f, interleaved))])
    latent = torch.cat([c, k_all], 1).double().numpy()
    for i in range(t):
        q = round_bf16(rope.rotate(qt[0, i].double().numpy(), np.full(128, at[i]), f, interleaved)).double().numpy()
        o, l = mla_oracle.attend_latent(qa[0, i].double().numpy(), q, latent[expanded.tree_sees(parents, t, i, n)], scale)
        assert np.abs(to[0, i].double().cpu().numpy() - o).max() <= 1e-2 * np.abs(o).max()
        assert np.abs(tl[0, i].double().cpu().numpy() - l).max() <= 1e-3
