"""The backward pass of the expanded form in 64 bits with torch, on any device, and what its roundings may amount to.
(The loops of the float64 oracle take minutes at the sizes of the GPU tests; test_backward_cpu.py holds this to them.)

Bounds, for a kernel that rounds p and ds to bf16 (half a step, 2^-8 of the value), sums in fp32 and rounds results to
bf16: a score's 192 products (fp32 sum: under 192 * 2^-24 of scale * sum|q||k|, 2^-11 on unit inputs: its exponential is off
by as much, relatively, which is counted as 2^-10); the difference d_out.v - delta has 128 products on each side, in fp32
under 2^-16 of sum|d_out||v| + sum|d_out||out| (+ 2^-23 |d_lse|, inside it).  So
    |dv|: (2^-8 + 2^-10) sum p|d_out|,   |ds| off by (2^-8 + 2^-10)|ds| + 2^-16 p (...) scale =: e,
    |dq|: sum e|k|,  |dk|: sum e|q|, and each result 2^-8 of itself more (and of the bound before it).
The fp32 sums over n rows add n * 2^-24 of the absolute sum: under 2^-11 of it for n <= 8192, inside the 2^-10.
"""
import torch


def backward(d, causal, scale, d_lse=None):
    """d: q_nope, q_rope, k_nope, k_rope, v, out, lse, d_out (any dtype), cu_q, cu_k (lists) -> gradients and bounds in
    64 bits, dicts by name; rows of no sequence are NaN."""
    dev = d["q_nope"].device
    f = dict(dtype=torch.float64, device=dev)
    nq, nk = d["q_nope"].shape[0], d["k_nope"].shape[0]
    g = dict(dq=torch.full((nq, 128, 192), float("nan"), **f), dk=torch.full((nk, 128, 128), float("nan"), **f),
             dr=torch.full((nk, 64), float("nan"), **f), dv=torch.full((nk, 128, 128), float("nan"), **f))
    b = {k: torch.zeros_like(v) for k, v in g.items()}
    cu_q, cu_k = [int(x) for x in d["cu_q"]], [int(x) for x in d["cu_k"]]
    for n in range(len(cu_q) - 1):
        qs, ks = slice(cu_q[n], cu_q[n + 1]), slice(cu_k[n], cu_k[n + 1])
        n_q, n_k = qs.stop - qs.start, ks.stop - ks.start
        see = torch.ones((n_q, n_k), dtype=torch.bool, device=dev)
        if causal:
            see = see.tril(n_k - n_q)
        g["dr"][ks] = 0
        for h in range(128):
            q = torch.cat((d["q_nope"][qs, h], d["q_rope"][qs, h]), -1).double()
            k = torch.cat((d["k_nope"][ks, h], d["k_rope"][ks]), -1).double()
            v, do, o = d["v"][ks, h].double(), d["d_out"][qs, h].double(), d["out"][qs, h].double()
            p = torch.exp(torch.where(see, scale * (q @ k.T) - d["lse"][qs, h].double()[:, None], -torch.inf))
            delta = (do * o).sum(-1, keepdim=True)
            if d_lse is not None:
                delta = delta - d_lse[qs, h].double()[:, None]
            ds = torch.where(see, p * (do @ v.T - delta), 0.0)
            e = (2.0 ** -8 + 2.0 ** -10) * ds.abs() + 2.0 ** -16 * p * (do.abs() @ v.abs().T + (do * o).abs().sum(-1, keepdim=True))
            ds, e = ds * scale, e * scale
            g["dq"][qs, h], b["dq"][qs, h] = ds @ k, e @ k.abs()
            dk, bk = ds.T @ q, e.T @ q.abs()
            g["dk"][ks, h], b["dk"][ks, h] = dk[:, :128], bk[:, :128]
            g["dr"][ks] += dk[:, 128:]
            b["dr"][ks] += bk[:, 128:]
            g["dv"][ks, h], b["dv"][ks, h] = p.T @ do, (2.0 ** -8 + 2.0 ** -10) * (p.T @ do.abs())

    def named(x):
        return dict(dq_nope=x["dq"][..., :128], dq_rope=x["dq"][..., 128:], dk_nope=x["dk"], dk_rope=x["dr"], dv=x["dv"])

    g = named(g)
    return g, {k: x + 2.0 ** -8 * (g[k].abs() + x) for k, x in named(b).items()}


NAMES = ("dq_nope", "dq_rope", "dk_nope", "dk_rope", "dv")


def check(got, d, causal, scale, d_lse=None, rows_q=None, rows_k=None):
    """Assert that the five gradients lie within the bounds (rows of sequences only)."""
    want, bound = backward(d, causal, scale, d_lse)
    for name, x in zip(NAMES, got):
        w, b = want[name].to(x.device), bound[name].to(x.device)
        inside = ~torch.isnan(w)
        off = (x.double() - w).abs()
        worst = torch.where(inside, off / b.clamp(min=1e-300), torch.zeros_like(off)).max().item() if x.numel() else 0.0
        ok = (off <= b) | ~inside | ((w == 0) & (x.double() == 0))
        assert bool(ok.all()), (name, worst, ok.logical_not().nonzero()[:4].tolist())
