"""The rotating append stores latents bit by bit as the plain append does, whatever they hold."""
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from oracle import rope

pytestmark = pytest.mark.gpu


def every_bf16(rows, width):
    """All 65,536 bit patterns (NaN payloads of both signs among them) over and over."""
    n = torch.arange(rows * width, dtype=torch.int32, device="cuda")
    return (n * 40503).bitwise_and(0xFFFF).sub(32768).to(torch.int16).view(torch.bfloat16).view(rows, width)


# one group of rows a CTA, and four
@pytest.mark.parametrize("rows", [1, 130, 8300])
def test_bf16_latents_are_stored_as_they_are(cuda_device, rows):
    pages = (rows + 63) // 64
    c, r = every_bf16(rows, 512), torch.randn((rows, 64), device="cuda").to(torch.bfloat16)
    table = torch.randperm(pages, device="cuda").to(torch.int32)[None].contiguous()
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([rows], [0, rows]))
    plain, rotated = (torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    binding.mla_cache_append_bf16(c, r, plain, table, lens, cu)
    binding.mla_cache_append_rope_bf16(c, r, binding.mla_rope_init(rope.frequencies()), rotated, table, lens, cu)
    assert torch.equal(rotated[..., :512].view(torch.int16), plain[..., :512].view(torch.int16))
    token = torch.arange(rows, device="cuda")
    stored = rotated[table[0, token // 64].long(), token % 64, :512]
    assert torch.equal(stored.view(torch.int16), c.view(torch.int16))


# groups that hold an infinity or a NaN, and values of every size
@pytest.mark.parametrize("fmt,width", [("fp8", 594), ("fp4", 324), ("fp8_v41", 528), ("fp4_v41", 288)])
@pytest.mark.parametrize("rows", [130, 8300])
def test_quantised_latents_are_the_plain_appends(cuda_device, fmt, width, rows):
    pages = (rows + 63) // 64
    g = torch.Generator(device="cuda").manual_seed(rows)
    size = torch.randint(-133, 127, (rows, 32, 1), generator=g, device="cuda").double()
    c = (torch.randn((rows, 32, 16), generator=g, device="cuda").double() * 2.0 ** size).view(rows, 512).to(torch.bfloat16)
    some = torch.rand((rows, 512), generator=g, device="cuda") < 0.002
    c[some] = every_bf16(rows, 512)[some]
    r = torch.randn((rows, 64), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([rows], [0, rows]))
    zero = torch.zeros(rows, dtype=torch.int32, device="cuda")      # position 0 turns nothing
    plain, rotated = (torch.zeros((pages, 64, width), dtype=torch.uint8, device="cuda") for _ in range(2))
    getattr(binding, "mla_cache_append_" + fmt)(c, r, plain, table, lens, cu)
    getattr(binding, "mla_cache_append_rope_" + fmt)(c, r, binding.mla_rope_init(rope.frequencies()), rotated, table, lens, cu,
                                                     positions=zero)
    assert torch.equal(rotated, plain)
