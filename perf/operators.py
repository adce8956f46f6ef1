"""Measured cases of the operators around the MLA decode: cache rows written and read, the expanded (prefill) form and
the attention of a drafted tree.

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
MAX_ROWS, MAX_EXPAND = 32768, 8192
MAX_PAIRS, MAX_KEYS = 32_000_000, 32768
MAX_NODE_TOKENS, MAX_CACHED = 2_000_000, 131072


# ---------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 sequences: each appends its new token's row (the smallest call: latency)
        {"name": "append bf16 step", "op": "append", "fmt": "bf16", "batch": 64, "new": 1, "ctx": 2048, "ragged": True,
         "lens_seed": 1},
        # a prompt of four ragged sequences quantised into the FP8 cache and read back
        {"name": "append fp8 prompt", "op": "append", "fmt": "fp8", "batch": 4, "new": 4096, "ctx": 0, "ragged": True,
         "lens_seed": 2},
        # the context of a chunked prefill read from an FP4 cache
        {"name": "gather fp4 context", "op": "gather", "fmt": "fp4", "batch": 2, "new": 16384, "ctx": 0, "ragged": False,
         "lens_seed": 3},
        # a short prompt's keys and values from its latent rows (ragged end: 130 rows)
        {"name": "expand 130", "op": "expand", "rows": 130},
        # a prefill chunk's worth of latent rows
        {"name": "expand 8192", "op": "expand", "rows": 8192},
        # a few very short prompts (latency; lengths one to a tile)
        {"name": "prefill short", "op": "prefill", "batch": 5, "new": 33, "ctx": 0, "ragged": True, "causal": True,
         "lens_seed": 4},
        # ragged prompts, as a serving batch holds them
        {"name": "prefill ragged", "op": "prefill", "batch": 8, "new": 2048, "ctx": 0, "ragged": True, "causal": True,
         "lens_seed": 5},
        # the next chunk of two long prompts over what is cached already
        {"name": "prefill chunk", "op": "prefill", "batch": 2, "new": 512, "ctx": 15000, "ragged": False, "causal": True,
         "lens_seed": 6},
        # one long prompt
        {"name": "prefill 8192", "op": "prefill", "batch": 1, "new": 8192, "ctx": 0, "ragged": False, "causal": True,
         "lens_seed": 7},
        # one sequence verifies eight drafted tokens (latency)
        {"name": "tree small", "op": "tree", "fmt": "bf16", "batch": 1, "nodes": 8, "ctx": 1000, "ragged": False,
         "lens_seed": 8},
        # a batch verifies trees of up to 16 nodes over ragged contexts
        {"name": "tree batch", "op": "tree", "fmt": "bf16", "batch": 16, "nodes": 16, "ctx": 8192, "ragged": True,
         "lens_seed": 9},
        # wide trees over the FP8 cache
        {"name": "tree fp8 wide", "op": "tree", "fmt": "fp8", "batch": 8, "nodes": 61, "ctx": 4096, "ragged": False,
         "lens_seed": 10},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(("append", "gather", "expand", "prefill", "prefill", "tree", "tree"))
    seed = rng.randrange(1 << 20)
    if op == "expand":
        return {"op": op, "rows": _log(rng, 1, MAX_EXPAND)}
    ragged = rng.random() < 0.7
    if op in ("append", "gather"):
        batch = _log(rng, 1, 128)
        new = _log(rng, 1, MAX_ROWS // batch)
        return {"op": op, "fmt": rng.choice(FORMATS), "batch": batch, "new": new,
                "ctx": _log(rng, 1, 4096) if op == "append" else 0, "ragged": ragged, "lens_seed": seed}
    if op == "prefill":
        batch = _log(rng, 1, 16)
        new = _log(rng, 1, 4096)
        new = max(1, min(new, math.isqrt(MAX_PAIRS // batch), MAX_KEYS // batch))
        ctx = 0 if rng.random() < 0.5 else _log(rng, 1, 16384)
        ctx = max(0, min(ctx, MAX_PAIRS // (batch * new) - new, MAX_KEYS // batch - new))
        return {"op": op, "batch": batch, "new": new, "ctx": ctx, "ragged": ragged, "causal": rng.random() < 0.8,
                "lens_seed": seed}
    batch = _log(rng, 1, 32)
    nodes = _log(rng, 1, 64)
    ctx = max(1, min(_log(rng, 1, 16384), MAX_NODE_TOKENS // (batch * nodes), MAX_CACHED // batch))
    return {"op": op, "fmt": rng.choice(FORMATS), "batch": batch, "nodes": nodes, "ctx": ctx, "ragged": ragged,
            "lens_seed": seed}


def _lens(case):
    """(new or node counts, context lengths) of the case's sequences."""
    r = random.Random(case["lens_seed"])
    top = case["nodes"] if case["op"] == "tree" else case["new"]
    n, ctx = [], []
    for _ in range(case["batch"]):
        n.append(r.randint(1, top) if case["ragged"] and top > 1 else top)
        ctx.append(r.randint(0, case["ctx"]) if case["ragged"] else case["ctx"])
    return n, ctx


def work(case):
    if case["op"] == "expand":
        n = case["rows"]
        return {"bytes": n * LATENT * 2 + 2 * HEADS * 128 * LATENT * 2 + 2 * n * HEADS * 128 * 2,
                "flops": 2 * n * LATENT * 2 * HEADS * 128}
    new, ctx = _lens(case)
    if case["op"] == "append":      # latent in, rows out; a quantised row is read back as bf16
        row = ROW_BYTES[case["fmt"]]
        return {"bytes": sum(new) * (1152 + row + (0 if case["fmt"] == "bf16" else row + 1152)), "flops": 0}
    if case["op"] == "gather":
        return {"bytes": sum(new) * (1152 + ROW_BYTES[case["fmt"]]), "flops": 0}
    if case["op"] == "prefill":
        keys = [a + c for a, c in zip(new, ctx)]
        pairs = sum(a * c + (a * (a + 1) // 2 if case["causal"] else a * a) for a, c in zip(new, ctx))
        return {"bytes": sum(new) * HEADS * (192 + 128) * 2 + sum(new) * HEADS * 4
                + sum(keys) * (HEADS * 256 + ROPE) * 2, "flops": 2 * pairs * HEADS * (192 + 128)}
    cached = sum(a + c for a, c in zip(new, ctx))
    seen = sum(a * (c + 1) for a, c in zip(new, ctx))       # at least its context and itself
    rows = case["batch"] * case["nodes"]
    return {"bytes": cached * ROW_BYTES[case["fmt"]] + sum(new) * HEADS * 576 * 2 + rows * HEADS * (512 * 2 + 4),
            "flops": 2 * seen * HEADS * (576 + 512)}


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


def _cache(fmt, pool, gen, filled):
    """A cache of `pool` pages; `filled`: every row holds a token's latent, else zeros."""
    dtype = torch.bfloat16 if fmt == "bf16" else torch.uint8
    width = 576 if fmt == "bf16" else ROW_BYTES[fmt]
    cache = torch.zeros((pool, PAGE, width), dtype=dtype, device="cuda")
    if filled:
        flat = cache.view(-1, width)
        for lo in range(0, flat.shape[0], 65536):
            n = min(65536, flat.shape[0] - lo)
            flat[lo:lo + n] = _encode(fmt, _normal(gen, n, LATENT), _normal(gen, n, ROPE))
    return cache


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    state = dict(case, workspace=torch.zeros(96 << 20, dtype=torch.uint8, device="cuda"))
    if op == "expand":
        # latent rows after their norm; weights of variance 1 / 512, as an initialised projection has
        state["latent"] = _normal(gen, case["rows"], LATENT + ROPE)
        state["w_uk"] = (torch.randn((HEADS, 128, LATENT), generator=gen, device="cuda") * LATENT ** -0.5).to(torch.bfloat16)
        state["w_uv"] = (torch.randn((HEADS, 128, LATENT), generator=gen, device="cuda") * LATENT ** -0.5).to(torch.bfloat16)
        return state
    new, ctx = _lens(case)
    total = sum(new)
    keys = [a + c for a, c in zip(new, ctx)]
    if op == "prefill":
        nk = sum(keys)
        q = _normal(gen, total, HEADS, 192)
        rows = _normal(gen, nk, LATENT + ROPE)              # gathered rows: their last 64 values are the keys' RoPE part
        state.update(q_nope=q[..., :128], q_rope=q[..., 128:], k_rope=rows[:, LATENT:], k_nope=_normal(gen, nk, HEADS, 128),
                     v=_normal(gen, nk, HEADS, 128), cu_q=_cu(new), cu_k=_cu(keys), host=(new, keys))
        return state
    table, pool = _pages(keys, gen)
    state.update(block_table=table, seq_lens=_ints(keys))
    if op == "tree":
        t = case["nodes"]
        # a node's parent is an earlier node, the latest ones more often, or the context (-1)
        at = torch.arange(t, device="cuda", dtype=torch.float32)
        back = torch.rand((case["batch"], t), generator=gen, device="cuda").square()
        parents = (at - 1 - torch.floor(back * (at + 1))).to(torch.int32).clamp_(min=-1)
        state.update(kv_cache=_cache(case["fmt"], pool, gen, True), parents=parents, n_nodes=_ints(new),
                     q_absorbed=_normal(gen, case["batch"], t, HEADS, LATENT),
                     q_rope=_normal(gen, case["batch"], t, HEADS, ROPE))
        return state
    state.update(cu_rows=_cu(new), n_rows=total, kv_cache=_cache(case["fmt"], pool, gen, op == "gather"))
    if op == "append":
        state.update(c_kv=_normal(gen, total, LATENT), k_rope=_normal(gen, total, ROPE))
    return state


# ---------------------------------------------------------------------------------------------------------- plain form
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantise(x, group, top, highest):
    """x [n, m] float32 -> (x / 2^k as float32, k + 127 as uint8), k the smallest integer with amax <= top 2^k."""
    g = x.view(x.shape[0], -1, group)
    m, e = torch.frexp(g.abs().amax(-1))
    ft, et = math.frexp(top)
    k = torch.where(m <= ft, e - et, e - et + 1)
    k = torch.where(m == 0, torch.zeros_like(k), k).clamp(-127, highest)
    scaled = torch.ldexp(g, -k.unsqueeze(-1)).clamp(-top, top)
    return scaled.reshape(x.shape), (k + 127).to(torch.uint8)


def _encode(fmt, c_kv, k_rope):
    """Cache rows of a format from latent and RoPE values (bf16)."""
    if fmt == "bf16":
        return torch.cat((c_kv, k_rope), -1)
    x = torch.cat((c_kv[:, :448] if fmt.endswith("v41") else c_kv, k_rope), -1).float()
    if fmt.startswith("fp8"):
        scaled, scales = _quantise(x, 32, 448.0, 119)
        return torch.cat((scaled.to(torch.float8_e4m3fn).view(torch.uint8), scales), -1)
    scaled, scales = _quantise(x, 16, 6.0, 125)
    a = scaled.abs()
    # to nearest, ties to the even code: the borders between the eight magnitudes, a tie going up to an even one
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + 8 * torch.signbit(scaled).to(torch.uint8)
    return torch.cat((code[:, 0::2] + 16 * code[:, 1::2], scales), -1)


def _decode(fmt, rows):
    """[n, width] cache rows -> [n, 576] float32."""
    if fmt == "bf16":
        return rows.float()
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


def _slots(block_table, seq_lens, cu_rows, n):
    """Cache slot of each packed row: row b's rows are the last of its seq_lens[b] tokens."""
    i = torch.arange(n, device=cu_rows.device)
    b = torch.searchsorted(cu_rows[1:], i.to(torch.int32), right=True)
    pos = seq_lens[b] - cu_rows[b + 1] + i
    return block_table[b, pos // PAGE].long() * PAGE + pos % PAGE


def _softmax(s):
    """(weights, log of the sum of exp) over the last axis; a row of -inf gives zeros and -inf."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total), (m + torch.log(total)).squeeze(-1)


def _plain_prefill(s):
    out = torch.empty((s["q_nope"].shape[0], HEADS, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((s["q_nope"].shape[0], HEADS), dtype=torch.float32, device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(*s["host"]):
        q = torch.cat((s["q_nope"][q0:q0 + nq], s["q_rope"][q0:q0 + nq]), -1).float().transpose(0, 1)
        rope = s["k_rope"][k0:k0 + nk].float().unsqueeze(0)
        see = torch.arange(nk, device="cuda") <= torch.arange(nq, device="cuda").unsqueeze(1) + (nk - nq)
        step = max(1, min(HEADS, (1 << 31) // (nq * nk)))   # heads at a time, so that the scores fit
        for h in range(0, HEADS, step):
            k = torch.cat((s["k_nope"][k0:k0 + nk, h:h + step].float().transpose(0, 1),
                           rope.expand(min(step, HEADS - h), nk, ROPE)), -1)
            x = torch.matmul(q[h:h + step], k.transpose(1, 2)).mul_(SCALE)
            if s["causal"]:
                x.masked_fill_(~see, -math.inf)
            p, l = _softmax(x)
            out[q0:q0 + nq, h:h + step] = torch.matmul(p, s["v"][k0:k0 + nk, h:h + step].float().transpose(0, 1)).transpose(0, 1)
            lse[q0:q0 + nq, h:h + step] = l.transpose(0, 1)
            del x, p
        q0, k0 = q0 + nq, k0 + nk
    return {"out": out, "lse": lse}


def _sees(parents):
    """[B, T, T]: node i sees node j, that is j is i or one of its ancestors."""
    t = parents.shape[1]
    see = torch.eye(t, dtype=torch.bool, device=parents.device).expand(parents.shape[0], t, t).clone()
    up = parents.long()
    for _ in range(t - 1):          # one step towards the root at a time
        see |= (torch.arange(t, device=parents.device) == up.unsqueeze(-1))
        up = torch.where(up >= 0, torch.gather(parents.long(), 1, up.clamp(min=0)), up)
    return see


def _plain_tree(s):
    b, t = s["parents"].shape
    q = torch.cat((s["q_absorbed"], s["q_rope"]), -1).float()
    if s["fmt"].endswith("v41"):
        q[..., 448:512] = 0
    out = torch.empty((b, t, HEADS, LATENT), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((b, t, HEADS), dtype=torch.float32, device="cuda")
    sees = _sees(s["parents"])
    longest = s["block_table"].shape[1] * PAGE
    flat = s["kv_cache"].view(-1, s["kv_cache"].shape[-1])
    pos = torch.arange(longest, device="cuda")
    node = torch.arange(t, device="cuda")
    for r in range(b):
        rows = _decode(s["fmt"], flat[s["block_table"][r].clamp(min=0).long()[pos // PAGE] * PAGE + pos % PAGE])
        ctx = s["seq_lens"][r] - s["n_nodes"][r]
        at = (pos - ctx).clamp(0, t - 1)
        see = (pos < ctx) | ((pos < s["seq_lens"][r]) & sees[r][:, at])
        see &= (node < s["n_nodes"][r]).unsqueeze(1)
        x = torch.matmul(q[r].view(t * HEADS, 576), rows.T).mul_(SCALE).view(t, HEADS, longest)
        p, l = _softmax(x.masked_fill_(~see.unsqueeze(1), -math.inf))
        out[r] = torch.matmul(p.view(t * HEADS, longest), rows[:, :LATENT]).view(t, HEADS, LATENT)
        lse[r] = l
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------------------------------------- one pass
def run(state):
    s, op = state, state["op"]
    if own:
        return _own(s, op)
    if op == "expand":
        c = s["latent"][:, :LATENT].float()
        w = torch.cat((s["w_uk"].view(-1, LATENT), s["w_uv"].view(-1, LATENT))).float()
        kv = torch.matmul(c, w.T).to(torch.bfloat16).view(-1, 2, HEADS, 128)
        return {"k_nope": kv[:, 0], "v": kv[:, 1]}
    if op == "prefill":
        return _plain_prefill(s)
    if op == "tree":
        return _plain_tree(s)
    at = _slots(s["block_table"], s["seq_lens"], s["cu_rows"], s["n_rows"])
    flat = s["kv_cache"].view(-1, s["kv_cache"].shape[-1])
    if op == "append":
        flat[at] = _encode(s["fmt"], s["c_kv"], s["k_rope"])
        if s["fmt"] == "bf16":
            return {"kv_cache": s["kv_cache"]}
    return {"rows": _decode(s["fmt"], flat[at]).to(torch.bfloat16)}


def _own(s, op):
    from mla_latent_kv_05_gb300 import binding
    ws = s["workspace"]
    if op == "expand":
        k, v = binding.mla_expand_kv(s["latent"][:, :LATENT], s["w_uk"], s["w_uv"], workspace=ws)
        return {"k_nope": k, "v": v}
    if op == "prefill":
        out, lse = binding.mla_prefill_bf16(s["q_nope"], s["q_rope"], s["k_nope"], s["k_rope"], s["v"], s["cu_q"],
                                            s["cu_k"], SCALE, causal=s["causal"], workspace=ws)
        return {"out": out, "lse": lse}
    if op == "tree":
        out, lse = getattr(binding, "mla_decode_tree_" + s["fmt"])(
            s["q_absorbed"], s["q_rope"], s["kv_cache"], s["block_table"], s["seq_lens"], s["parents"], SCALE,
            n_nodes=s["n_nodes"], workspace=ws)
        return {"out": out, "lse": lse}
    if op == "append":
        getattr(binding, "mla_cache_append_" + s["fmt"])(s["c_kv"], s["k_rope"], s["kv_cache"], s["block_table"],
                                                         s["seq_lens"], s["cu_rows"], workspace=ws)
        if s["fmt"] == "bf16":
            return {"kv_cache": s["kv_cache"]}
    # a quantised row is returned as the values it stands for
    return {"rows": getattr(binding, "mla_cache_gather_" + s["fmt"])(s["kv_cache"], s["block_table"], s["seq_lens"],
                                                                     s["cu_rows"], s["n_rows"], workspace=ws)}


# ---------------------------------------------------------------------------------------------------------- in 64 bits
def _exact_values(fmt, raw):
    """Cache bytes [n, width] (or bf16 rows) -> float64 [n, 576], from the formats' bit fields."""
    if fmt == "bf16":
        return raw.double()
    values = 512 if "v41" in fmt else 576
    raw = raw.long()
    if fmt.startswith("fp8"):
        c = raw[:, :values]
        e, f = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * torch.exp2((e - 7).double()))
        x, scale, group = torch.where(c >= 128, -mag, mag), raw[:, values:], 32
    else:
        c = raw[:, :values // 2].repeat_interleave(2, 1)
        c = torch.where(torch.arange(values, device=raw.device) % 2 == 0, c & 15, c >> 4)
        e, f = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(e == 0, f * 0.5, (1 + f / 2) * torch.exp2((e - 1).double()))
        x, scale, group = torch.where(c >= 8, -mag, mag), raw[:, values // 2:], 16
    x = x * torch.exp2((scale - 127).double()).repeat_interleave(group, 1)
    full = torch.zeros((raw.shape[0], 576), dtype=torch.float64, device=raw.device)
    full[:, :values - 64] = x[:, :values - 64]
    full[:, 512:] = x[:, values - 64:]
    return full


def _exact_rounded(fmt, c_kv, k_rope):
    """What the cache stands for after c_kv, k_rope are written to it, float64 [n, 576]."""
    full = torch.cat((c_kv, k_rope), -1).double()
    if fmt == "bf16":
        return full
    if "v41" in fmt:
        full[:, 448:512] = 0
    group, top, mantissa, lowest = (32, 448.0, 3, -6) if fmt.startswith("fp8") else (16, 6.0, 1, 0)
    x = full.view(full.shape[0], -1, group)
    k = torch.ceil(torch.log2(x.abs().amax(-1, keepdim=True) / top))
    k = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
    a = x / torch.exp2(k)
    binade = torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -60))).clamp(min=lowest)
    step = torch.exp2(binade - mantissa)
    return (torch.round(a / step) * step * torch.exp2(k)).view(full.shape)


def _exact_attend(q, k, v, see):
    """q [h, n, d], k [h, m, d], v [h, m, e] float64, see [n, m] -> out [h, n, e], lse [h, n]."""
    x = (q @ k.transpose(-1, -2)) * SCALE
    x = torch.where(see, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1)
    p = torch.where(see, torch.exp(x - torch.where(lse == -math.inf, torch.zeros_like(lse), lse).unsqueeze(-1)), torch.zeros_like(x))
    return p @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "expand":
        c = s["latent"][:, :LATENT].double()
        return {"k_nope": torch.einsum("nc,hdc->nhd", c, s["w_uk"].double()),
                "v": torch.einsum("nc,hdc->nhd", c, s["w_uv"].double())}
    new, ctx = _lens(case)
    if op == "prefill":
        outs, lses = [], []
        q0 = k0 = 0
        for nq, c in zip(new, ctx):
            nk = nq + c
            see = torch.ones((nq, nk), dtype=torch.bool, device="cuda")
            if case["causal"]:
                see = see.tril(c)
            q = torch.cat((s["q_nope"][q0:q0 + nq], s["q_rope"][q0:q0 + nq]), -1).double()
            heads = []
            for h in range(HEADS):
                k = torch.cat((s["k_nope"][k0:k0 + nk, h], s["k_rope"][k0:k0 + nk]), -1).double()
                heads.append(_exact_attend(q[:, h], k, s["v"][k0:k0 + nk, h].double(), see))
            outs.append(torch.stack([o for o, _ in heads], 1))
            lses.append(torch.stack([l for _, l in heads], 1))
            q0, k0 = q0 + nq, k0 + nk
        return {"out": torch.cat(outs), "lse": torch.cat(lses)}
    table = s["block_table"].cpu().tolist()
    flat = s["kv_cache"].view(-1, s["kv_cache"].shape[-1])

    def slots(b, lo, hi):
        return torch.tensor([table[b][j // PAGE] * PAGE + j % PAGE for j in range(lo, hi)], dtype=torch.long, device="cuda")

    if op == "tree":
        t = case["nodes"]
        out = torch.zeros((case["batch"], t, HEADS, LATENT), dtype=torch.float64, device="cuda")
        lse = torch.full((case["batch"], t, HEADS), -math.inf, dtype=torch.float64, device="cuda")
        parents = s["parents"].cpu().tolist()
        for b, (n, c) in enumerate(zip(new, ctx)):
            rows = _exact_values(case["fmt"], flat[slots(b, 0, n + c)])
            for i in range(n):
                seen, up = list(range(c)), i
                while up >= 0:
                    seen.append(c + up)
                    up = parents[b][up]
                k = rows[torch.tensor(seen, device="cuda")]
                q = torch.cat((s["q_absorbed"][b, i], s["q_rope"][b, i]), -1).double()
                see = torch.ones((HEADS, len(seen)), dtype=torch.bool, device="cuda")
                out[b, i], lse[b, i] = _exact_attend(q, k, k[:, :LATENT], see)
        return {"out": out, "lse": lse}
    at = torch.cat([slots(b, c, c + n) for b, (n, c) in enumerate(zip(new, ctx))])
    if op == "gather":
        return {"rows": _exact_values(case["fmt"], flat[at])}
    rows = _exact_rounded(case["fmt"], s["c_kv"], s["k_rope"])
    if case["fmt"] == "bf16":
        cache = s["kv_cache"].double()
        cache.view(-1, 576)[at] = rows
        return {"kv_cache": cache}
    return {"rows": rows}
