"""Inputs and outputs that end where the mapped memory ends: TMA maps claim nothing behind a tensor."""
import ctypes

import pytest
import torch

from mla_latent_kv_05_gb300 import binding

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


class Memory:
    """An allocation of its own (not the caching allocator's), whose last bytes tensors are placed on."""

    def __init__(self, nbytes):
        self.rt = ctypes.CDLL("libcudart.so")
        self.ptr, self.n = ctypes.c_void_p(0), nbytes
        torch.cuda.synchronize()
        assert self.rt.cudaMalloc(ctypes.byref(self.ptr), ctypes.c_size_t(nbytes)) == 0
        self.__cuda_array_interface__ = dict(shape=(nbytes // 2,), typestr="<i2", data=(self.ptr.value, False), version=3)
        self.flat = torch.as_tensor(self, device="cuda").view(torch.bfloat16)
        assert self.flat.data_ptr() == self.ptr.value

    def last(self, x):
        """A copy of x whose last byte is the allocation's."""
        t = self.flat[self.flat.numel() - x.numel():].view(x.shape)
        t.copy_(x)
        return t

    def free(self):
        torch.cuda.synchronize()
        assert self.rt.cudaFree(self.ptr) == 0


@pytest.fixture
def memory(cuda_device):
    m = Memory(2 << 20)
    yield m
    m.free()


@pytest.mark.parametrize("width", [64, 576])
@pytest.mark.parametrize("n", [1, 81, 200, 400])
def test_prefill_with_keys_at_the_end(memory, n, width):
    g = torch.Generator(device="cuda").manual_seed(n)
    q, rows = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16) for s in ((n, 128, 192), (n, width)))
    k, v = (torch.randn((n, 128, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    want = binding.mla_prefill_bf16(q[..., :128], q[..., 128:], k, rows[:, width - 64:], v, cu, cu, SCALE)
    got = binding.mla_prefill_bf16(q[..., :128], q[..., 128:], k, memory.last(rows)[:, width - 64:], v, cu, cu, SCALE)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("n", [1, 3, 8])
def test_prefill_with_short_queries_and_values_at_the_end(memory, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    q, k, v, kr = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
                   for s in ((n, 128, 192), (n, 128, 128), (n, 128, 128), (n, 64)))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    want = binding.mla_prefill_bf16(q[..., :128], q[..., 128:], k, kr, v, cu, cu, SCALE)
    for i in range(3):
        a = [q, k, v]
        a[i] = memory.last(a[i])
        got = binding.mla_prefill_bf16(a[0][..., :128], a[0][..., 128:], a[1], kr, a[2], cu, cu, SCALE)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("n", [1, 33, 100, 300])
def test_expand_with_latents_and_results_at_the_end(memory, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    rows = torch.randn((n, 576), generator=g, device="cuda").to(torch.bfloat16)
    w = [(torch.randn((128, 128, 512), generator=g, device="cuda") * 512 ** -0.5).to(torch.bfloat16) for _ in range(2)]
    want = binding.mla_expand_kv(rows[:, :512], *w)
    got = binding.mla_expand_kv(memory.last(rows)[:, :512], *w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    if n <= 33:
        k = memory.last(torch.zeros((n, 128, 128), dtype=torch.bfloat16, device="cuda"))
        got = binding.mla_expand_kv(rows[:, :512], *w, k_nope=k)
        assert got[0] is k and all(torch.equal(a, b) for a, b in zip(got, want))


def test_tree_with_queries_at_the_end(memory):
    g = torch.Generator(device="cuda").manual_seed(1)
    qa, qr, cache = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
                     for s in ((1, 3, 128, 512), (1, 3, 128, 64), (2, 64, 576)))
    table, lens, parents = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[1, 0]], [100], [[-1, 0, 0]]))
    want = binding.mla_decode_tree_bf16(qa, qr, cache, table, lens, parents, SCALE)
    got = binding.mla_decode_tree_bf16(qa, memory.last(qr), cache, table, lens, parents, SCALE)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
