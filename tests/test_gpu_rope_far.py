"""The rotating append at positions past 2^18: the bytes of vectors rotated by the table's own fractions of a turn (exact in
integers), which are within |position| 2^-65 turns of the frequencies'."""
import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import binding
from oracle import rope, row_codec
from test_gpu_rope import FORMATS, Cache, round_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("fmt", list(FORMATS))
def test_bytes_at_far_positions(cuda_device, fmt, interleaved):
    s = Cache([200, 57], [30, 0], seed=50)
    f = rope.frequencies(factor=40.0)
    table = binding.mla_rope_init(f, interleaved=interleaved)
    pos = torch.randint(-2 ** 31, 2 ** 31, (s.n,), generator=s.g).to(torch.int32)
    pos[:8] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 18, 2 ** 22 + 1, -1, 2 ** 24 + 1, 2 ** 30, -2 ** 20])
    got = s.append(fmt, table, positions=pos.cuda())
    units = np.array([[int(p) * int(u) % 2 ** 64 for u in table.turns] for p in pos], dtype=object)
    # 64-bit fractions as angles in [0, 2 pi), known to 2^-50
    angle = 2 * np.pi * (units / 2 ** 64).astype(np.float64)
    x, y = s.r[:s.n].double().numpy(), np.empty((s.n, 64))
    a, b = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    y[:, a], y[:, b] = x[:, a] * np.cos(angle) - x[:, b] * np.sin(angle), x[:, a] * np.sin(angle) + x[:, b] * np.cos(angle)
    want = s.empty(fmt).cpu().view(-1, FORMATS[fmt])
    if fmt == "bf16":
        want[s.slots] = torch.cat([s.c[:s.n], round_bf16(y)], 1)
    else:
        want[s.slots] = torch.from_numpy(row_codec.encode_rows(s.c[:s.n].double().numpy(), y, fmt))
    assert torch.equal(got.cpu().view(-1, FORMATS[fmt]), want)
    # and the frequencies' angles: 2^-65 turns a position are 2^-62.3 radians, and the float64 product's rounding of the
    # largest angles, 2^31 times 1, is 2^-22
    far = np.abs(pos.double().numpy())[:, None]
    off = np.abs(np.exp(1j * angle) - np.exp(1j * pos.double().numpy()[:, None] * np.asarray(f)))
    assert (off <= far * (2.0 ** -62 + 2.0 ** -52) + 2.0 ** -48).all()
