"""The operators around the decode on several streams and in captured graphs:
every result is the bits of the same call made alone."""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from mla_latent_kv_05_gb300 import inputs as gen

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Tree:
    def __init__(self, fmt, seed):
        inp = gen.make_inputs(3, 7, [60 + 31 * seed, 500, 129], kv_dtype=fmt, seed=seed)
        self.args = [x.cuda() for x in (inp.q_absorbed, inp.q_rope, inp.kv_cache, inp.block_table, inp.seq_lens)]
        self.parents = torch.arange(-1, 6, dtype=torch.int32, device="cuda").repeat(3, 1)
        self.fn = getattr(binding, "mla_decode_tree_" + fmt)
        self.ws = binding.alloc_workspace_tree(3, 7, max_pages=inp.max_pages if fmt != "bf16" else 0)
        self.scale = inp.scale

    def __call__(self, stream=None, ws=None):
        return self.fn(*self.args, self.parents, self.scale, workspace=self.ws if ws is None else ws, stream=stream)


class Prefill:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        n = 300 + 70 * seed

        def r(*shape):
            return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()

        self.q, self.qr, self.kr = r(n, 128, 128), r(n, 128, 64), r(n, 64)
        self.latent, self.w = r(n, 512), (r(128, 128, 512) * 512 ** -0.5, r(128, 128, 512) * 512 ** -0.5)
        self.cu = ints(0, n // 3, n)
        self.ws, self.ews = binding.alloc_workspace_prefill(2, n), torch.zeros(256, dtype=torch.uint8, device="cuda")

    def __call__(self, stream=None, ws=None):
        k, v = binding.mla_expand_kv(self.latent, *self.w, workspace=self.ews, stream=stream)
        return binding.mla_prefill_bf16(self.q, self.qr, k, self.kr, v, self.cu, self.cu, SCALE,
                                        workspace=self.ws if ws is None else ws, stream=stream)


class Rows:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.c, self.r = (torch.randn((700, m), generator=g).to(torch.bfloat16).cuda() for m in (512, 64))
        self.cache = torch.zeros((12, 64, 594), dtype=torch.uint8, device="cuda")
        self.at = torch.randperm(12, generator=g).to(torch.int32)[None].cuda().contiguous(), ints(700), ints(0, 700)
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def __call__(self, stream=None, ws=None):
        binding.mla_cache_append_fp8(self.c, self.r, self.cache, *self.at, workspace=self.ws, stream=stream)
        rows = binding.mla_cache_gather_fp8(self.cache, *self.at, 700, workspace=self.ws, stream=stream)
        return self.cache, rows


def calls():
    return [Tree("bf16", 1), Tree("fp8", 2), Prefill(1), Prefill(3), Rows(4), Tree("fp4", 3)]


def test_calls_on_streams_at_once(cuda_device):
    todo = calls()
    want = [[x.clone() for x in c()] for c in todo]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in todo]
    got = []
    for _ in range(3):
        got = []
        for c, s in zip(todo, streams):
            with torch.cuda.stream(s):                  # outputs belong to the stream that fills them
                got.append(c(stream=s))
    torch.cuda.synchronize()
    for c, a, b in zip(todo, got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b)), type(c).__name__
        assert binding.mla_get_status(c.ws) == 0


def test_two_graphs_that_share_a_workspace(cuda_device):
    for pair in ((Tree("bf16", 1), Tree("fp8", 2)), (Prefill(1), Prefill(3))):
        want = [[x.clone() for x in c()] for c in pair]
        ws = max((c.ws for c in pair), key=lambda w: w.numel())
        graphs, outs = [], []
        for c in pair:
            c(ws=ws)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(c(ws=ws))
            graphs.append(g)
        for k in (0, 1, 1, 0, 1, 0):
            for x in outs[k]:
                x.fill_(float("nan"))
            graphs[k].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(outs[k], want[k])), (type(pair[0]).__name__, k)
        assert binding.mla_get_status(ws) == 0
