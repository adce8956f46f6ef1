"""Rotary positions without a GPU: the oracle's pins, the table's arithmetic, and what the entry points refuse."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from mla_latent_kv_05_gb300 import _build, binding
from oracle import rope

# pi to 60 digits
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


# ------------------------------------------------------------------ oracle
@pytest.mark.parametrize("interleaved", [True, False])
def test_the_oracle_turns_pairs_as_complex_numbers(interleaved):
    rng = np.random.default_rng(1)
    x, pos, f = rng.standard_normal((7, 3, 64)), rng.integers(0, 10 ** 5, 7), rope.frequencies()
    z = x[..., 0::2] + 1j * x[..., 1::2] if interleaved else x[..., :32] + 1j * x[..., 32:]
    want = z * np.exp(1j * np.outer(pos, f))[:, None, :]
    y = rope.rotate(x, pos, f, interleaved)
    got = y[..., 0::2] + 1j * y[..., 1::2] if interleaved else y[..., :32] + 1j * y[..., 32:]
    assert np.abs(got - want).max() < 1e-9
    # and back
    assert np.abs(rope.rotate(y, pos, f, interleaved, inverse=True) - x).max() < 1e-9


def test_products_of_rotated_vectors_depend_on_the_distance_alone():
    rng = np.random.default_rng(2)
    q, k, f = rng.standard_normal((1, 64)), rng.standard_normal((1, 64)), rope.frequencies(factor=40.0)
    a = rope.rotate(q, [100], f, True) @ rope.rotate(k, [37], f, True).T
    b = rope.rotate(q, [5100], f, True) @ rope.rotate(k, [5037], f, True).T
    assert abs(a - b).max() < 1e-9


def test_scaled_frequencies_by_hand():
    f, g = rope.frequencies(), rope.frequencies(factor=40.0)
    # 64 ln(4096 / (2 pi 32)) / (2 ln 10^4) = 10.47, with 1 in place of 32: 22.51
    for i in range(32):
        if i <= 10:
            assert g[i] == f[i]
        elif i >= 23:
            assert g[i] == pytest.approx(f[i] / 40, rel=1e-15)
        else:
            t = (i - 10) / 13
            assert g[i] == pytest.approx(f[i] / 40 * t + f[i] * (1 - t), rel=1e-14)


# ------------------------------------------------------------------ host functions
@pytest.mark.parametrize("kw", [{}, dict(factor=40.0), dict(base=500000.0, factor=8.0, original_tokens=8192),
                                dict(factor=4.0, original_tokens=64, beta_fast=8.0, beta_slow=2.0)])
def test_frequencies_are_the_oracles(lib, kw):
    want = rope.frequencies(**{("original" if k == "original_tokens" else k): v for k, v in kw.items()})
    # a power and a logarithm, each off by a few units of the last place
    assert binding.mla_rope_frequencies(**kw) == pytest.approx(want, rel=1e-13)


@pytest.mark.parametrize("f", [rope.frequencies(), [0.0] * 32, [-(0.5 ** i) for i in range(32)],
                               [1024.0 - i * math.pi for i in range(32)], [2 * math.pi] * 32])
def test_the_table_is_the_fraction_of_a_turn_to_its_last_bit(lib, f):
    table = binding.mla_rope_init(f, scale=0.5, interleaved=False)
    assert table.scale == 0.5 and table.interleaved == 0
    for got, x in zip(table.turns, f):
        want = Fraction(x) / (2 * PI) * 2 ** 64
        off = (got - want) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        # half a unit, and what the two-part 1 / (2 pi) loses (2^-107 of it) and fma's rounding of the rest
        assert off <= Fraction(1, 2) + abs(Fraction(x)) * Fraction(1, 2 ** 40)


def test_host_functions_refuse(lib):
    with pytest.raises(ValueError):
        binding.mla_rope_init([1.0] * 31)
    for bad in (float("nan"), float("inf"), 1025.0, -1e9):
        with pytest.raises(binding.MLAError):
            binding.mla_rope_init([bad] + [1.0] * 31)
    with pytest.raises(binding.MLAError):
        binding.mla_rope_init([1.0] * 32, scale=float("nan"))
    for kw in (dict(base=1.0), dict(base=float("nan")), dict(factor=0.5), dict(factor=float("inf")),
               dict(original_tokens=0), dict(beta_slow=0.0), dict(beta_fast=1.0, beta_slow=1.0),
               dict(beta_fast=float("inf"))):
        with pytest.raises(binding.MLAError):
            binding.mla_rope_frequencies(**kw)


def table():
    return binding.mla_rope_init(rope.frequencies())


def test_rope_entry_refuses_on_the_host(lib):
    fake, z = ctypes.c_void_p(0x1000), ctypes.c_void_p(0)
    t = table()
    at = ctypes.addressof(t)

    def call(x=fake, strides=(8192, 64, 8192, 64), positions=fake, rows=4, heads=128, rope_at=at, out=fake):
        return lib.mla_rope_bf16(x, (ctypes.c_size_t * 4)(*strides), positions, rows, heads, rope_at, 0, out, z)

    assert call(x=z) == -1 and call(positions=z) == -1 and call(out=z) == -1 and call(rope_at=None) == -1
    assert call(rows=-1) == -1 and call(heads=-1) == -1
    assert call(rows=(1 << 24) + 1) == -2 and call(heads=4097) == -2
    for i in range(4):
        for bad in (0, 12, 1 << 40):
            s = [8192, 64, 8192, 64]
            s[i] = bad
            assert call(strides=s) == -1
    assert call(x=ctypes.c_void_p(0x1008)) == -1 and call(out=ctypes.c_void_p(0x1002)) == -1
    assert call(positions=ctypes.c_void_p(0x1002)) == -1
    assert call(strides=(8192, 64, 8192, 128)) == -1 and call(strides=(8192, 64, 16384, 64)) == -1     # in place, elsewhere
    assert call(rows=0) == 0 and call(heads=0) == 0
    t.scale = float("inf")
    assert call() == -1


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "fp4", "fp8_v41", "fp4_v41"])
def test_append_entries_refuse_on_the_host(lib, fmt):
    fn = getattr(lib, "mla_cache_append_rope_" + fmt)
    fake, z = ctypes.c_void_p(0x1000), ctypes.c_void_p(0)
    t = table()

    def call(c=fake, cs=512, r=fake, rs=64, positions=z, at=ctypes.addressof(t), cache=fake, tbl=fake, batch=2, rows=4,
             pages=8, page=64, max_pages=4, ws=fake, n=256):
        return fn(c, cs, r, rs, positions, at, cache, tbl, fake, fake, batch, rows, pages, page, max_pages, ws, n, z)

    for kw in (dict(c=z), dict(r=z), dict(at=None), dict(cache=z), dict(tbl=z), dict(ws=z), dict(cs=0), dict(rs=12),
               dict(batch=-1), dict(rows=-1), dict(pages=0), dict(max_pages=0), dict(positions=ctypes.c_void_p(0x1002)),
               dict(cache=ctypes.c_void_p(0x1008)), dict(c=ctypes.c_void_p(0x1008))):
        assert call(**kw) == -1, kw
    assert call(page=32) == -2 and call(batch=1 << 17) == -2
    assert call(n=8) == -3
    assert call(rows=0) == 0 and call(batch=0) == 0


def test_the_binding_refuses_what_is_not_a_table_or_not_vectors():
    x, p = torch.zeros((4, 128, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.mla_rope_bf16(x, p, table())                       # not on a CUDA device
    with pytest.raises(ValueError):
        binding.mla_rope_bf16(x[0, 0], p, table())                 # one vector without its row
    with pytest.raises(TypeError):
        binding.mla_rope_bf16(None, p, table())
    with pytest.raises(TypeError):
        binding._rope_arg({"turns": []})
