"""Measured cases of the rotary positions, the cache append that rotates on the way, and the backward pass of the
expanded (prefill) attention.

`run` computes a pass in plain torch operations where `own` is false, and through this package's entry points where it
is true.  A case's sequence lengths follow from its own numbers (`lens_seed`); everything else comes from the seed."""
import math
import random

import torch

own = False

HEADS, LATENT, ROPE, PAGE = 128, 512, 64, 64
SCALE = 1.0 / math.sqrt(128 + 64)
# bytes of one cached token
ROW_BYTES = {"bf16": 1152, "fp8": 594, "fp4": 324, "fp8_v41": 528, "fp4_v41": 288}
FORMATS = ("bf16", "fp8", "fp4", "fp8_v41", "fp4_v41")
# sizes that bound a drawn case: those of the largest listed ones
MAX_VECTORS, MAX_ROWS = 8192 * HEADS, 16384
MAX_PAIRS, MAX_QUERIES, MAX_KEYS = 4096 * 4096, 8192, 16384
LONGEST = 163840        # tokens of the longest context: 40 times 4096


# ---------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the queries of one decode step of 64 sequences (latency)
        {"name": "rope step", "op": "rope", "rows": 64, "heads": 128, "width": 64, "interleaved": True, "yarn": False,
         "inverse": False, "packed": False},
        # a long prompt's queries, the last 64 values of 192-value heads, with positions scaled for long contexts
        {"name": "rope prompt", "op": "rope", "rows": 8192, "heads": 128, "width": 192, "interleaved": True, "yarn": True,
         "inverse": False, "packed": True},
        # a training step's gradient of rotated queries, back to the unrotated ones; half layout, odd row count
        {"name": "rope gradient", "op": "rope", "rows": 1523, "heads": 128, "width": 64, "interleaved": False,
         "yarn": False, "inverse": True, "packed": True},
        # one decode step of 64 sequences: each appends its new token's row (the smallest call: latency)
        {"name": "append bf16 step", "op": "append", "fmt": "bf16", "batch": 64, "new": 1, "ctx": 2048, "ragged": True,
         "interleaved": True, "yarn": False, "tree": False, "lens_seed": 21},
        # sixteen sequences append sixteen drafted nodes each: positions that are not the rows' places in the cache
        {"name": "append fp8 nodes", "op": "append", "fmt": "fp8", "batch": 16, "new": 16, "ctx": 8192, "ragged": True,
         "interleaved": True, "yarn": True, "tree": True, "lens_seed": 22},
        # a prompt of four ragged sequences rotated and quantised into the FP8 cache, and read back
        {"name": "append fp8 prompt", "op": "append", "fmt": "fp8", "batch": 4, "new": 4096, "ctx": 0, "ragged": True,
         "interleaved": True, "yarn": True, "tree": False, "lens_seed": 23},
        # the next chunk of two long prompts into the FP4 cache of 288-byte rows; half layout
        {"name": "append fp4 chunk", "op": "append", "fmt": "fp4_v41", "batch": 2, "new": 4001, "ctx": 15000,
         "ragged": False, "interleaved": False, "yarn": True, "tree": False, "lens_seed": 24},
        # a few very short sequences (latency; lengths one to a tile)
        {"name": "backward short", "op": "backward", "batch": 5, "new": 33, "ctx": 0, "ragged": True, "causal": True,
         "dlse": False, "lens_seed": 25},
        # a packed training batch of ragged sequences
        {"name": "backward ragged", "op": "backward", "batch": 8, "new": 1024, "ctx": 0, "ragged": True, "causal": True,
         "dlse": False, "lens_seed": 26},
        # full attention over three sequences of an odd length
        {"name": "backward full", "op": "backward", "batch": 3, "new": 777, "ctx": 0, "ragged": False, "causal": False,
         "dlse": False, "lens_seed": 27},
        # the last chunk of two long sequences, whose parts are merged by their LSE: the LSE has a gradient too
        {"name": "backward chunk", "op": "backward", "batch": 2, "new": 512, "ctx": 7500, "ragged": False, "causal": True,
         "dlse": True, "lens_seed": 28},
        # one long training sequence
        {"name": "backward 4096", "op": "backward", "batch": 1, "new": 4096, "ctx": 0, "ragged": False, "causal": True,
         "dlse": False, "lens_seed": 29},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(("rope", "rope", "append", "append", "backward", "backward", "backward"))
    seed = rng.randrange(1 << 20)
    if op == "rope":
        heads = rng.choice((1, 16, 128, 128))
        return {"op": op, "rows": _log(rng, 1, MAX_VECTORS // 128), "heads": heads, "width": rng.choice((64, 192)),
                "interleaved": rng.random() < 0.5, "yarn": rng.random() < 0.5, "inverse": rng.random() < 0.4,
                "packed": rng.random() < 0.5}
    ragged = rng.random() < 0.7
    if op == "append":
        batch = _log(rng, 1, 128)
        new = _log(rng, 1, MAX_ROWS // batch)
        return {"op": op, "fmt": rng.choice(FORMATS), "batch": batch, "new": new, "ctx": _log(rng, 1, 8192),
                "ragged": ragged, "interleaved": rng.random() < 0.5, "yarn": rng.random() < 0.5,
                "tree": new <= 64 and rng.random() < 0.5, "lens_seed": seed}
    batch = _log(rng, 1, 16)
    new = _log(rng, 1, 4096)
    new = max(1, min(new, MAX_QUERIES // batch, math.isqrt(MAX_PAIRS // batch)))
    ctx = 0 if rng.random() < 0.6 else _log(rng, 1, 8192)
    ctx = max(0, min(ctx, MAX_PAIRS // (batch * new) - new, MAX_KEYS // batch - new))
    return {"op": op, "batch": batch, "new": new, "ctx": ctx, "ragged": ragged, "causal": rng.random() < 0.8,
            "dlse": rng.random() < 0.3, "lens_seed": seed}


def _lens(case):
    """(new, context) lengths of the case's sequences."""
    r = random.Random(case["lens_seed"])
    n, ctx = [], []
    for _ in range(case["batch"]):
        n.append(r.randint(1, case["new"]) if case["ragged"] and case["new"] > 1 else case["new"])
        ctx.append(r.randint(0, case["ctx"]) if case["ragged"] else case["ctx"])
    return n, ctx


def work(case):
    if case["op"] == "rope":
        n = case["rows"]
        return {"bytes": n * 4 + 2 * n * case["heads"] * ROPE * 2, "flops": 0}
    new, ctx = _lens(case)
    if case["op"] == "append":      # latent in, rows out; a quantised row is read back as bf16
        row = ROW_BYTES[case["fmt"]]
        return {"bytes": sum(new) * (1152 + row + (0 if case["fmt"] == "bf16" else row + 1152)), "flops": 0}
    keys = [a + c for a, c in zip(new, ctx)]
    pairs = sum(a * c + (a * (a + 1) // 2 if case["causal"] else a * a) for a, c in zip(new, ctx))
    # queries and their gradients, out and its gradient, lse; keys, values and their gradients
    return {"bytes": sum(new) * HEADS * (2 * 192 * 2 + 2 * 128 * 2 + 4 + (4 if case["dlse"] else 0))
            + sum(keys) * (HEADS * 256 + ROPE) * 2 * 2, "flops": 2 * pairs * HEADS * (3 * 192 + 2 * 128)}


# ---------------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cu(counts):
    total, out = 0, [0]
    for c in counts:
        total += c
        out.append(total)
    return _ints(out)


def _pages(seq_lens, gen):
    """A page table over a shuffled pool, and the pool's size."""
    need = [(s + PAGE - 1) // PAGE for s in seq_lens]
    pool = max(1, sum(need)) + 3
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    width = max(1, max(need))
    row = torch.repeat_interleave(torch.arange(len(need), device="cuda"), torch.tensor(need, device="cuda"))
    start = torch.tensor([sum(need[:b]) for b in range(len(need))], device="cuda")
    col = torch.arange(sum(need), device="cuda") - start[row]
    table = torch.full((len(need), width), -1, dtype=torch.int32, device="cuda")
    table[row, col] = perm[:sum(need)]
    return table, pool


def _frequencies(yarn):
    """Radians a token of the 32 pairs: 10000^(-i/32), or these scaled for 40 times 4096 tokens: pairs that turn 32 times
    or more over 4096 tokens stay, those that turn less than once are slowed 40-fold, with a ramp between."""
    f = [10000.0 ** (-i / 32) for i in range(32)]
    if not yarn:
        return f
    low, high = (64 * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0)) for turns in (32.0, 1.0))
    low, high = max(math.floor(low), 0), min(math.ceil(high), 63)
    ramp = [min(max((i - low) / (high - low), 0.0), 1.0) for i in range(32)]
    return [x / 40.0 * r + x * (1.0 - r) for x, r in zip(f, ramp)]


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    state = dict(case)
    if op != "backward":
        state["freq"] = _frequencies(case["yarn"])
    if op == "rope":
        rows, longest = case["rows"], LONGEST if case["yarn"] else 4096
        # a packed row's positions run on from a start; a decode step's rows are each somewhere else
        if case["packed"]:
            start = torch.randint(0, max(1, longest - rows), (1,), generator=gen, device="cuda")
            state["positions"] = (start + torch.arange(rows, device="cuda")).to(torch.int32)
        else:
            state["positions"] = torch.randint(0, longest, (rows,), generator=gen, device="cuda").to(torch.int32)
        state["x"] = _normal(gen, rows, case["heads"], case["width"])[..., case["width"] - ROPE:]
    else:
        new, ctx = _lens(case)
        keys = [a + c for a, c in zip(new, ctx)]
        if op == "append":
            table, pool = _pages(keys, gen)
            quantised = case["fmt"] != "bf16"
            state.update(block_table=table, seq_lens=_ints(keys), cu_rows=_cu(new), n_rows=sum(new), positions=None,
                         c_kv=_normal(gen, sum(new), LATENT), k_rope=_normal(gen, sum(new), ROPE),
                         kv_cache=torch.zeros((pool, PAGE, ROW_BYTES[case["fmt"]] if quantised else 576),
                                              dtype=torch.uint8 if quantised else torch.bfloat16, device="cuda"))
            if case["tree"]:
                # a drafted node stands at most as deep as its number says
                n = torch.tensor(new, device="cuda")
                at = torch.arange(sum(new), device="cuda") - torch.repeat_interleave(torch.cumsum(n, 0) - n, n)
                depth = torch.floor(torch.rand(sum(new), generator=gen, device="cuda") * (at + 1)).long()
                state["positions"] = (torch.repeat_interleave(torch.tensor(ctx, device="cuda"), n) + depth).to(torch.int32)
        else:
            nq, nk = sum(new), sum(keys)
            q = _normal(gen, nq, HEADS, 192)
            rows = _normal(gen, nk, LATENT + ROPE)          # gathered rows: their last 64 values are the keys' RoPE part
            state.update(q_nope=q[..., :128], q_rope=q[..., 128:], k_rope=rows[:, LATENT:], k_nope=_normal(gen, nk, HEADS, 128),
                         v=_normal(gen, nk, HEADS, 128), cu_q=_cu(new), cu_k=_cu(keys), host=(new, keys))
            state["out"], state["lse"] = _plain_forward(state)
            state["d_out"] = _normal(gen, nq, HEADS, 128)
            state["d_lse"] = torch.randn((nq, HEADS), generator=gen, device="cuda") if case["dlse"] else None
    if own:
        _handles(state)
    return state


# ---------------------------------------------------------------------------------------------------------- plain form
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _rotate(x, positions, freq, interleaved, inverse):
    """x [rows, heads, 64] rotated in 64 bits (angles of far positions)."""
    angle = positions.double().unsqueeze(1) * torch.tensor(freq, dtype=torch.float64, device=x.device)
    c, s = torch.cos(angle).unsqueeze(1), torch.sin(angle).unsqueeze(1)
    if inverse:
        s = -s
    x = x.double()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    a, b = a * c - b * s, a * s + b * c
    return torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)


def _power(k):
    """2^k in 64 bits, from its bits (a library's power may be off by a rounding, which matters at a tie)."""
    return (k.long() + 1023 << 52).view(torch.float64)


def _quantise(x, group, top, mantissa, lowest, highest):
    """x [n, m] float64 -> (x / 2^k rounded to the format's values, k + 127 as uint8), k the smallest integer with
    amax <= top 2^k."""
    g = x.view(x.shape[0], -1, group)
    m, e = torch.frexp(g.abs().amax(-1))
    ft, et = math.frexp(top)
    k = torch.where(m <= ft, e - et, e - et + 1)
    k = torch.where(m == 0, torch.zeros_like(k), k).clamp(-127, highest)
    scaled = (g * _power(-k).unsqueeze(-1)).clamp(-top, top)
    # to nearest, ties to even: in 64 bits, because a rotated value may lie next to a border
    step = _power((torch.frexp(scaled)[1] - 1).clamp(min=lowest) - mantissa)
    return (torch.round(scaled / step) * step).reshape(x.shape), (k + 127).to(torch.uint8)


def _encode(fmt, c_kv, k_rope):
    """Cache rows of a format from latent (bf16) and rotated values (float64)."""
    if fmt == "bf16":
        return torch.cat((c_kv, k_rope.to(torch.bfloat16)), -1)
    x = torch.cat((c_kv[:, :448] if fmt.endswith("v41") else c_kv, k_rope), -1)
    if fmt.startswith("fp8"):
        scaled, scales = _quantise(x, 32, 448.0, 3, -6, 119)
        return torch.cat((scaled.to(torch.float8_e4m3fn).view(torch.uint8), scales), -1)
    scaled, scales = _quantise(x, 16, 6.0, 1, 0, 125)
    code = torch.searchsorted(torch.tensor(E2M1, dtype=torch.float64, device=x.device), scaled.abs().contiguous())
    code = (code + 8 * torch.signbit(scaled)).to(torch.uint8)
    return torch.cat((code[:, 0::2] + 16 * code[:, 1::2], scales), -1)


def _decode(fmt, rows):
    """[n, width] quantised cache rows -> [n, 576] float32."""
    values = 512 if fmt.endswith("v41") else 576
    if fmt.startswith("fp8"):
        x, scales, group = rows[:, :values].contiguous().view(torch.float8_e4m3fn).float(), rows[:, values:], 32
    else:
        b = rows[:, :values // 2].to(torch.int64)
        code = torch.stack((b & 15, b >> 4), -1).view(rows.shape[0], values)
        x = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)[code]
        scales, group = rows[:, values // 2:], 16
    x = torch.ldexp(x.view(rows.shape[0], -1, group), scales.to(torch.int32).unsqueeze(-1) - 127).view(rows.shape[0], values)
    if values == 576:
        return x
    return torch.cat((x[:, :448], torch.zeros_like(x[:, :64]), x[:, 448:]), -1)


def _places(block_table, seq_lens, cu_rows, n):
    """Token index and cache slot of each packed row: row b's rows are the last of its seq_lens[b] tokens."""
    i = torch.arange(n, device=cu_rows.device)
    b = torch.searchsorted(cu_rows[1:], i.to(torch.int32), right=True)
    pos = seq_lens[b] - cu_rows[b + 1] + i
    return pos, block_table[b, pos // PAGE].long() * PAGE + pos % PAGE


def _parts(s):
    """For each sequence and run of heads: slices of queries, keys and heads, q, k, v [heads, n, d] in 32 bits, and which
    pairs are seen (None: all)."""
    q0 = k0 = 0
    for nq, nk in zip(*s["host"]):
        qs, ks = slice(q0, q0 + nq), slice(k0, k0 + nk)
        see = None
        if s["causal"]:
            see = torch.arange(nk, device="cuda") <= torch.arange(nq, device="cuda").unsqueeze(1) + (nk - nq)
        step = max(1, min(HEADS, (1 << 30) // (nq * nk)))   # heads at a time, so that the scores fit
        for h in range(0, HEADS, step):
            hs = slice(h, min(HEADS, h + step))
            q = torch.cat((s["q_nope"][qs, hs], s["q_rope"][qs, hs]), -1).float().transpose(0, 1)
            rope = s["k_rope"][ks].float().unsqueeze(0).expand(hs.stop - h, nk, ROPE)
            k = torch.cat((s["k_nope"][ks, hs].float().transpose(0, 1), rope), -1)
            yield qs, ks, hs, q, k, s["v"][ks, hs].float().transpose(0, 1), see
        q0, k0 = q0 + nq, k0 + nk


def _plain_forward(s):
    """The attention's output and LSE, which its backward pass takes."""
    out = torch.empty((s["q_nope"].shape[0], HEADS, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((s["q_nope"].shape[0], HEADS), dtype=torch.float32, device="cuda")
    for qs, ks, hs, q, k, v, see in _parts(s):
        x = torch.matmul(q, k.transpose(1, 2)).mul_(SCALE)
        if see is not None:
            x.masked_fill_(~see, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = x.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        out[qs, hs] = torch.matmul(p, v).div_(total).transpose(0, 1).to(torch.bfloat16)
        lse[qs, hs] = (m + torch.log(total)).squeeze(-1).transpose(0, 1)
        del x, p
    return out, lse


def _plain_backward(s):
    nq, nk = s["q_nope"].shape[0], s["k_nope"].shape[0]
    new = dict(dtype=torch.bfloat16, device="cuda")
    dq = torch.empty((nq, HEADS, 192), **new)
    dk, dv = torch.empty((nk, HEADS, 128), **new), torch.empty((nk, HEADS, 128), **new)
    dk_rope = torch.zeros((nk, ROPE), dtype=torch.float32, device="cuda")
    for qs, ks, hs, q, k, v, see in _parts(s):
        do = s["d_out"][qs, hs].float().transpose(0, 1)
        p = torch.matmul(q, k.transpose(1, 2)).mul_(SCALE).sub_(s["lse"][qs, hs].transpose(0, 1).unsqueeze(-1)).exp_()
        if see is not None:
            p.masked_fill_(~see, 0.0)
        dv[ks, hs] = torch.matmul(p.transpose(1, 2), do).transpose(0, 1).to(torch.bfloat16)
        delta = (do * s["out"][qs, hs].float().transpose(0, 1)).sum(-1, keepdim=True)
        if s["d_lse"] is not None:
            delta = delta - s["d_lse"][qs, hs].transpose(0, 1).unsqueeze(-1)
        ds = torch.matmul(do, v.transpose(1, 2)).sub_(delta).mul_(p).mul_(SCALE)
        del p
        dq[qs, hs] = torch.matmul(ds, k).transpose(0, 1).to(torch.bfloat16)
        g = torch.matmul(ds.transpose(1, 2), q)
        dk[ks, hs] = g[..., :128].transpose(0, 1).to(torch.bfloat16)
        dk_rope[ks] += g[..., 128:].sum(0)
        del ds, g
    return {"dq_nope": dq[..., :128], "dq_rope": dq[..., 128:], "dk_nope": dk, "dk_rope": dk_rope.to(torch.bfloat16), "dv": dv}


# ---------------------------------------------------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["op"]
    if own:
        return _own(s, op)
    if op == "rope":
        return {"y": _rotate(s["x"], s["positions"], s["freq"], s["interleaved"], s["inverse"]).to(torch.bfloat16)}
    if op == "backward":
        return _plain_backward(s)
    pos, at = _places(s["block_table"], s["seq_lens"], s["cu_rows"], s["n_rows"])
    if s["positions"] is not None:
        pos = s["positions"]
    flat = s["kv_cache"].view(-1, s["kv_cache"].shape[-1])
    k = _rotate(s["k_rope"].unsqueeze(1), pos, s["freq"], s["interleaved"], False).squeeze(1)
    flat[at] = _encode(s["fmt"], s["c_kv"], k)
    if s["fmt"] == "bf16":
        return {"kv_cache": s["kv_cache"]}
    return {"rows": _decode(s["fmt"], flat[at]).to(torch.bfloat16)}


def _handles(s):
    """What a user's program keeps from call to call: the rotation's table, and a workspace."""
    from mla_latent_kv_05_gb300 import binding
    if s["op"] == "backward":
        s["workspace"] = binding.alloc_workspace_prefill_backward(len(s["host"][0]), s["q_nope"].shape[0], s["k_nope"].shape[0])
        return
    s["rope"] = binding.mla_rope_init(s["freq"], interleaved=s["interleaved"])
    s["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")


def _own(s, op):
    from mla_latent_kv_05_gb300 import binding
    if "workspace" not in s:
        _handles(s)
    if op == "rope":
        return {"y": binding.mla_rope_bf16(s["x"], s["positions"], s["rope"], inverse=s["inverse"])}
    if op == "backward":
        names = ("dq_nope", "dq_rope", "dk_nope", "dk_rope", "dv")
        return dict(zip(names, binding.mla_prefill_backward_bf16(
            s["d_out"], s["q_nope"], s["q_rope"], s["k_nope"], s["k_rope"], s["v"], s["out"], s["lse"], s["cu_q"],
            s["cu_k"], SCALE, causal=s["causal"], d_lse=s["d_lse"], workspace=s["workspace"])))
    getattr(binding, "mla_cache_append_rope_" + s["fmt"])(
        s["c_kv"], s["k_rope"], s["rope"], s["kv_cache"], s["block_table"], s["seq_lens"], s["cu_rows"],
        positions=s["positions"], workspace=s["workspace"])
    if s["fmt"] == "bf16":
        return {"kv_cache": s["kv_cache"]}
    # a quantised row is returned as the values it stands for
    return {"rows": getattr(binding, "mla_cache_gather_" + s["fmt"])(s["kv_cache"], s["block_table"], s["seq_lens"],
                                                                     s["cu_rows"], s["n_rows"], workspace=s["workspace"])}


# ---------------------------------------------------------------------------------------------------------- in 64 bits
def _exact_rotation(x, positions, freq, interleaved, inverse):
    """The pairs as complex numbers, turned by e^(i angle)."""
    z = x.double()
    z = z.unflatten(-1, (32, 2)) if interleaved else z.unflatten(-1, (2, 32)).transpose(-1, -2)
    turn = torch.outer(positions.double(), torch.tensor(freq, dtype=torch.float64, device=x.device))
    turn = torch.polar(torch.ones_like(turn), -turn if inverse else turn)
    while turn.dim() < z.dim() - 1:
        turn = turn.unsqueeze(1)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
    return z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)


def _exact_rounded(fmt, full):
    """What quantised rows stand for after `full` [n, 576] is written to them."""
    if "v41" in fmt:
        full[:, 448:512] = 0
    group, top, mantissa, lowest = (32, 448.0, 3, -6) if fmt.startswith("fp8") else (16, 6.0, 1, 0)
    x = full.view(full.shape[0], -1, group)
    amax = x.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(amax / top))
    k = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
    # (the logarithm of a power of two may come out next to the integer)
    k = torch.where((amax > 0) & (amax <= top * torch.exp2(k - 1)), k - 1, k)
    k = torch.where(amax > top * torch.exp2(k), k + 1, k)
    a = x / torch.exp2(k)
    binade = torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -60)))
    binade = torch.where(a.abs() < torch.exp2(binade), binade - 1, binade)
    binade = torch.where(a.abs() >= torch.exp2(binade + 1), binade + 1, binade).clamp(min=lowest)
    step = torch.exp2(binade - mantissa)
    return (torch.round(a / step) * step * torch.exp2(k)).view(full.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"y": _exact_rotation(s["x"], s["positions"], s["freq"], case["interleaved"], case["inverse"])}
    new, ctx = _lens(case)
    if case["op"] == "append":
        table = s["block_table"].cpu().tolist()
        tokens = [(b, c + i) for b, (n, c) in enumerate(zip(new, ctx)) for i in range(n)]
        at = torch.tensor([table[b][t // PAGE] * PAGE + t % PAGE for b, t in tokens], dtype=torch.long, device="cuda")
        pos = s["positions"] if case["tree"] else torch.tensor([t for _, t in tokens], device="cuda")
        full = torch.cat((s["c_kv"].double(), _exact_rotation(s["k_rope"], pos, s["freq"], case["interleaved"], False)), -1)
        if case["fmt"] != "bf16":
            return {"rows": _exact_rounded(case["fmt"], full)}
        cache = s["kv_cache"].double()
        cache.view(-1, 576)[at] = full
        return {"kv_cache": cache}
    f = {"dtype": torch.float64, "device": "cuda"}
    nq, nk = sum(new), sum(new) + sum(ctx)
    dq, dk, dv = torch.zeros((nq, HEADS, 192), **f), torch.zeros((nk, HEADS, 192), **f), torch.zeros((nk, HEADS, 128), **f)
    q0 = k0 = 0
    for n, c in zip(new, ctx):
        m = n + c
        unseen = torch.ones((n, m), dtype=torch.bool, device="cuda").triu(c + 1) if case["causal"] else None
        for h in range(HEADS):
            q = torch.cat((s["q_nope"][q0:q0 + n, h], s["q_rope"][q0:q0 + n, h]), -1).double()
            k = torch.cat((s["k_nope"][k0:k0 + m, h], s["k_rope"][k0:k0 + m]), -1).double()
            v, do = s["v"][k0:k0 + m, h].double(), s["d_out"][q0:q0 + n, h].double()
            x = SCALE * (q @ k.T) - s["lse"][q0:q0 + n, h].double().unsqueeze(1)
            if unseen is not None:
                x = x.masked_fill(unseen, -math.inf)
            p = torch.exp(x)
            # out is an input: the gradient through the softmax's normalisation is its product with d_out
            through = torch.einsum("nd,nd->n", do, s["out"][q0:q0 + n, h].double())
            if case["dlse"]:
                through = through - s["d_lse"][q0:q0 + n, h].double()
            g = SCALE * p * (do @ v.T - through.unsqueeze(1))
            dq[q0:q0 + n, h], dk[k0:k0 + m, h], dv[k0:k0 + m, h] = g @ k, g.T @ q, p.T @ do
        q0, k0 = q0 + n, k0 + m
    return {"dq_nope": dq[..., :128], "dq_rope": dq[..., 128:], "dk_nope": dk[..., :128], "dk_rope": dk[..., 128:].sum(1), "dv": dv}
