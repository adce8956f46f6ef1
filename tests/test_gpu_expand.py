"""The expansion of latent rows into keys and values on the GPU against a
float64 product.  Bound per element: the bf16 result's rounding (2^-8 of the
value) plus the fp32 accumulation of 512 products (512 steps of at most 2^-24
of sum |c||w|, doubled: 2^-14)."""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding

pytestmark = pytest.mark.gpu


def make(n, seed, stride=512):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn((n, stride), generator=g).to(torch.bfloat16).cuda()
    w = [(torch.randn((128, 128, 512), generator=g) * 512 ** -0.5).to(torch.bfloat16).cuda() for _ in range(2)]
    return rows, w[0], w[1]


def check(got, c, w):
    c, w = c.double(), w.double()
    ref = torch.einsum("nc,hdc->nhd", c, w)
    mag = torch.einsum("nc,hdc->nhd", c.abs(), w.abs())
    err = (got.double() - ref).abs()
    assert bool((err <= 2.0 ** -8 * ref.abs() + 2.0 ** -14 * mag).all()), float(err.max())


@pytest.mark.parametrize("n", [1, 7, 64, 127, 128, 129, 300, 1000, 2500])
def test_matches_float64(cuda_device, n):
    rows, w_uk, w_uv = make(n, n)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    k, v = binding.mla_expand_kv(rows, w_uk, w_uv, workspace=ws)
    assert binding.mla_get_status(ws) == 0
    check(k, rows, w_uk)
    check(v, rows, w_uv)


@pytest.mark.parametrize("n", [8192 + 257, 16900])
def test_more_tokens_than_a_block_of_tiles_on_sampled_rows(cuda_device, n):
    rows, w_uk, w_uv = make(n, n)
    k, v = binding.mla_expand_kv(rows, w_uk, w_uv)
    at = torch.cat([torch.arange(0, n, 509), torch.tensor([8191, 8192, 8193, n - 257, n - 1])]).cuda()
    check(k[at], rows[at], w_uk)
    check(v[at], rows[at], w_uv)


def test_strided_rows_outputs_given_and_neighbours_kept(cuda_device):
    rows, w_uk, w_uv = make(200, 3, 576)
    k = torch.full((202, 128, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full((202, 128, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    a, b = binding.mla_expand_kv(rows[:, :512], w_uk, w_uv, k_nope=k[1:201], v=v[1:201])
    assert a.data_ptr() == k[1:201].data_ptr()
    check(a, rows[:, :512], w_uk)
    check(b, rows[:, :512], w_uv)
    for t in (k, v):
        assert bool((t[0] == 5).all()) and bool((t[201] == 5).all())


def test_captured_and_replayed_on_another_stream(cuda_device):
    rows, w_uk, w_uv = make(140, 4)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    k, v = binding.mla_expand_kv(rows, w_uk, w_uv, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        binding.mla_expand_kv(rows, w_uk, w_uv, k_nope=k, v=v, workspace=ws)
    rows.copy_(make(140, 5)[0])
    g.replay()
    torch.cuda.synchronize()
    assert binding.mla_get_status(ws) == 0
    check(k, rows, w_uk)
    check(v, rows, w_uv)


def test_nothing_to_do(cuda_device):
    rows, w_uk, w_uv = make(1, 6)
    k, v = binding.mla_expand_kv(rows[:0], w_uk, w_uv)
    assert k.shape == (0, 128, 128) and v.shape == (0, 128, 128)
